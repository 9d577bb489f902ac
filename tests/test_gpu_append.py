"""GPU tests of art_rope_append against its 64-bit definition.

A rotated value is x cos - y sin in fp32: cosine and sine are off by at most
2^-22 (the angle's 2^-32 of a turn, the leading bits' conversion, sincospi,
and the amplitude's product), each product and the sum by 2^-24 of their sizes,
then one rounding to the stored type (bf16 2^-8 relative at most half a step
being 2^-9; 2^-8 is allowed).  So |error| <= 2^-21 (|x| + |y|) * amplitude
(+ 2^-8 |value|).  Unrotated channels, values and all other rows are copies."""
import math

import numpy as np
import pytest
import torch

from tests import cache_ref as ref

pytestmark = pytest.mark.gpu


def freqs(rot, base=10000.0):
    return base ** (-2.0 * np.arange(rot // 2) / max(rot, 1))


def close(got, x, want, rot, layout, amplitude):
    y = x.double()
    mag = torch.zeros_like(y)
    i = slice(0, rot // 2) if layout == "half" else slice(0, rot, 2)
    j = slice(rot // 2, rot) if layout == "half" else slice(1, rot, 2)
    mag[..., i] = mag[..., j] = y[..., i].abs() + y[..., j].abs()
    tol = 2.0 ** -21 * mag * abs(amplitude)
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * want.abs() * (mag > 0)
    err = (got.double().cpu() - want).abs()
    assert bool((err <= tol).all()), f"off by {float((err - tol).max()):.3g}"


def run(art, *, dtype="bf16", Hq=8, Hkv=2, d=128, rot=None, layout="half", page=16, B=3, lens=(5, 40, 1), start=(0, 7, 100),
        positions=None, amplitude=1.0, mass=True, pad=True, seed=0, in_place=False, rope=None, f=None, padded=0):
    rot = d if rot is None else rot
    g = torch.Generator().manual_seed(seed)
    width = max(-(-(s + n) // page) for s, n in zip(start, lens)) + 1
    k, v, table = ref.paged([s + n for s, n in zip(start, lens)], page, Hkv, d, dtype, seed, stale=3.0, width=width)
    seq = torch.cat([torch.full((n,), b) for b, n in enumerate(lens)])
    slot = torch.cat([torch.arange(s, s + n) for s, n in zip(start, lens)])
    if pad:            # padding tokens at both ends and inside
        seq = torch.cat([torch.tensor([-1]), seq[:2], torch.tensor([0]), seq[2:], torch.tensor([-1])])
        slot = torch.cat([torch.tensor([4]), slot[:2], torch.tensor([-1]), slot[2:], torch.tensor([-5])])
    T = len(seq)
    order = torch.randperm(T, generator=g)       # tokens of a batch in any order
    seq, slot = seq[order].int(), slot[order].int()
    pos = slot if positions is None else torch.as_tensor(positions(T), dtype=torch.int32)
    q, kn, vn = (torch.randn(T, h, d + padded, generator=g).to(ref.DT[dtype])[..., padded:] for h in (Hq, Hkv, Hkv))
    f = freqs(rot) if f is None else f
    rope = art.art_rope_init(d, rot_dim=rot, layout=layout, amplitude=amplitude) if rope is None else rope
    dev = "cuda"
    kc, vc = k.to(dev), v.to(dev)
    m0 = torch.rand(B, Hkv, width * page, generator=g)
    m = m0.to(dev) if mass else None
    status = torch.zeros(1, dtype=torch.int32, device=dev)

    def on_gpu(x):
        base = torch.empty(*x.shape[:-1], d + padded, dtype=x.dtype, device=dev)[..., padded:]
        return base.copy_(x)

    qg = on_gpu(q)
    out = torch.full((T, Hq, d), 9.0, dtype=q.dtype, device=dev)
    got = art.art_rope_append(rope, qg, on_gpu(kn), on_gpu(vn), kc, vc, table.to(dev), slot.to(dev),
                              positions=None if positions is None else pos.to(dev), token_seq=seq.to(dev), mass=m,
                              q_out=qg if in_place else out, device_status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    live = ((seq >= 0) & (slot >= 0)).nonzero().flatten()
    dead = ((seq < 0) | (slot < 0)).nonzero().flatten()
    cos, sin = ref.turn_by(f, pos.numpy(), amplitude)
    qw, kw = (ref.rotate(x, cos, sin, rot, layout) for x in (q, kn))
    close(got[live.to(dev)].cpu(), q[live], qw[live], rot, layout, amplitude)
    assert torch.equal(got[dead.to(dev)].cpu(), q[dead] if in_place else torch.full_like(q[dead], 9.0))
    assert torch.equal(got[..., rot:][live.to(dev)].cpu(), q[..., rot:][live])
    pg, row = table[seq[live].long(), slot[live].long() // page].long(), slot[live].long() % page
    close(kc.cpu()[pg, :, row], kn[live], kw[live], rot, layout, amplitude)
    assert torch.equal(kc.cpu()[pg, :, row][..., rot:], kn[live][..., rot:])
    v[pg, :, row] = vn[live]
    assert torch.equal(vc.cpu(), v)
    kc2 = kc.cpu()
    kc2[pg, :, row] = k[pg, :, row]
    assert torch.equal(kc2, k)                   # no other row of K changed
    if mass:
        m0[seq[live].long(), :, slot[live].long()] = 0.0
        assert torch.equal(m.cpu(), m0)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,rot", [(64, 64), (128, 128), (128, 32), (128, 6), (96, 96), (96, 40), (256, 64), (16, 2), (64, 0)])
def test_layouts_and_partial_rotation(cuda_lib, layout, dtype, d, rot):
    run(cuda_lib, dtype=dtype, d=d, rot=rot, layout=layout, seed=d + rot)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,rot", [(128, 100), (128, 102), (16, 14), (48, 26), (80, 20), (144, 142), (256, 250), (256, 8)])
def test_rotated_part_of_no_whole_vectors(cuda_lib, layout, dtype, d, rot):
    run(cuda_lib, dtype=dtype, d=d, rot=rot, layout=layout, seed=d + rot, Hq=9, Hkv=3)
    run(cuda_lib, dtype=dtype, d=d, rot=rot, layout=layout, seed=d + rot, in_place=True, mass=False)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("padded", [0, 3])
@pytest.mark.parametrize("rot", [0, 6, 32, 50])
def test_channels_behind_the_rotated_ones_keep_their_bits(cuda_lib, layout, dtype, padded, rot):
    """Infinities, NaN payloads and signed zeros among them, beside rotated ones in a vector."""
    art, dev, d, page = cuda_lib, "cuda", 64, 16
    bits = torch.int16 if dtype == "bf16" else torch.int32
    special = [0x7f80, 0xff80 - 0x10000, 0x7fc5, 0xff95 - 0x10000, 0, -0x8000, 0x0001, 0x3f80]
    special = torch.tensor(special, dtype=torch.int32)
    special = special.to(bits) if dtype == "bf16" else (special << 16) | 3
    g = torch.Generator().manual_seed(rot)

    def rows(h):
        base = torch.randn(5, h, d + padded, generator=g).to(ref.DT[dtype])
        x = base[..., padded:]
        x.view(bits)[..., rot:] = special[torch.randint(8, (5, h, d - rot), generator=g)]
        return x, base.to(dev)[..., padded:]

    (q, qg), (k, kg), (v, vg) = rows(3), rows(2), rows(2)
    kc = torch.zeros(1, 2, page, d, dtype=q.dtype, device=dev)
    vc = torch.zeros_like(kc)
    out = art.art_rope_append(art.art_rope_init(d, rot_dim=rot, layout=layout), qg, kg, vg, kc, vc,
                              torch.zeros(1, 1, dtype=torch.int32, device=dev), torch.arange(5, dtype=torch.int32, device=dev),
                              token_seq=torch.zeros(5, dtype=torch.int32, device=dev))
    kept = kc[0, :, :5].transpose(0, 1).contiguous().cpu()
    assert torch.equal(out.cpu().contiguous().view(bits)[..., rot:], q.contiguous().view(bits)[..., rot:])
    assert torch.equal(kept.view(bits)[..., rot:], k.contiguous().view(bits)[..., rot:])
    assert torch.equal(vc[0, :, :5].transpose(0, 1).contiguous().cpu().view(bits), v.contiguous().view(bits))
    assert bool(torch.isfinite(out[..., :rot].float()).all())


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (28, 4), (5, 5), (71, 1)])
def test_head_counts(cuda_lib, Hq, Hkv):
    run(cuda_lib, Hq=Hq, Hkv=Hkv)


@pytest.mark.parametrize("page", [1, 5, 64])
def test_page_sizes(cuda_lib, page):
    run(cuda_lib, page=page)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_far_and_negative_positions(cuda_lib, dtype):
    far = [0, 1, -1, 131071, 10 ** 6 + 1, 2 ** 31 - 1, -2 ** 31, 123456789, -131071]
    run(cuda_lib, dtype=dtype, positions=lambda T: [far[i % len(far)] for i in range(T)])


def test_in_place_queries(cuda_lib):
    run(cuda_lib, in_place=True)
    run(cuda_lib, in_place=True, layout="interleaved", rot=36)


def test_many_tokens(cuda_lib):
    run(cuda_lib, B=2, lens=(3000, 4097), start=(0, 50), page=64, Hq=6, Hkv=2, mass=False)


@pytest.mark.parametrize("padded", [8, 3])
def test_strided_rows(cuda_lib, padded):
    """Rows on 16-byte boundaries, and rows that are not (scalar path)."""
    run(cuda_lib, padded=padded)
    run(cuda_lib, padded=padded, dtype="f32", layout="interleaved")


def test_broadcast_values(cuda_lib):
    """k and v expanded over the heads (stride 0) are read as they are."""
    art, dev = cuda_lib, "cuda"
    g = torch.Generator().manual_seed(2)
    k, v, table = ref.paged([10], 16, 4, 64, "bf16", 1, stale=0.0)
    kn, vn, q = (torch.randn(1, 1, 64, generator=g).to(torch.bfloat16) for _ in range(3))
    kc, vc = k.to(dev), v.to(dev)
    rope = art.art_rope_init(64)
    art.art_rope_append(rope, q.to(dev).expand(1, 8, 64), kn.to(dev).expand(1, 4, 64), vn.to(dev).expand(1, 4, 64), kc, vc,
                        table.to(dev), torch.tensor([10], dtype=torch.int32, device=dev))
    torch.cuda.synchronize()
    pg = int(table[0, 0])
    assert torch.equal(vc.cpu()[pg, :, 10], vn[0].expand(4, 64))
    assert bool((kc[pg, :, 10] == kc[pg, :1, 10]).all())


def test_scalings(cuda_lib):
    """linear, ntk and by_parts against their formulas, with an amplitude; given frequencies."""
    art, rot, base, L0, s = cuda_lib, 128, 10000.0, 4096, 8.0
    f = freqs(rot, base)
    run(art, rope=art.art_rope_init(128, base=base, scaling="linear", factor=s), f=f / s)
    run(art, rope=art.art_rope_init(128, base=base, scaling="ntk", factor=s), f=freqs(rot, base * s ** (rot / (rot - 2))))
    turns = L0 * f / (2 * math.pi)
    keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0, 1)
    amp = 0.1 * math.log(s) + 1
    run(art, rope=art.art_rope_init(128, base=base, scaling="by_parts", factor=s, original_len=L0, amplitude=amp),
        f=keep * f + (1 - keep) * f / s, amplitude=amp, positions=lambda T: [1000 * i for i in range(T)])
    odd = [2.5, -0.25, 0.0, 7.0 * math.pi, 1e-9, 3.0]
    run(art, rot=12, rope=art.art_rope_init(128, rot_dim=12, inv_freq=odd), f=np.array(odd))


def test_turning_back_restores(cuda_lib):
    """Positions p and then -p: the rotation undone, to twice its rounding."""
    art, dev = cuda_lib, "cuda"
    g = torch.Generator().manual_seed(3)
    k, v, table = ref.paged([8], 16, 2, 64, "f32", 1, stale=0.0)
    q, kn, vn = torch.randn(1, 4, 64, generator=g), torch.randn(1, 2, 64, generator=g), torch.randn(1, 2, 64, generator=g)
    rope = art.art_rope_init(64, layout="interleaved")
    slot = torch.tensor([9], dtype=torch.int32, device=dev)
    x = q.to(dev)
    for p in (99999, -99999):
        x = art.art_rope_append(rope, x, kn.to(dev), vn.to(dev), k.to(dev), v.to(dev), table.to(dev), slot,
                                positions=torch.tensor([p], dtype=torch.int32, device=dev))
    torch.cuda.synchronize()
    pair = q.view(1, 4, 32, 2).abs().sum(-1, keepdim=True).expand(1, 4, 32, 2).reshape(1, 4, 64)
    assert bool(((x.cpu() - q).abs() <= 2.0 ** -19 * pair).all())


def test_out_of_range_tokens_are_reported_and_skipped(cuda_lib):
    art, dev = cuda_lib, "cuda"
    k, v, table = ref.paged([40, 40], 16, 2, 64, "bf16", 1, stale=0.0)
    bad_table = table.clone()
    bad_table[1, 0] = k.shape[0]
    q, kn, vn = (torch.ones(1, h, 64, dtype=torch.bfloat16, device=dev) for h in (4, 2, 2))
    rope = art.art_rope_init(64)
    for seq, slot, tb in ((2, 0, table), (0, 48, table), (0, 2 ** 31 - 1, table), (1, 3, bad_table), (0, 45, table)):
        kc, vc = k.to(dev), v.to(dev)
        status = torch.zeros(1, dtype=torch.int32, device=dev)
        out = torch.full_like(q, 9.0)
        art.art_rope_append(rope, q, kn, vn, kc, vc, tb.to(dev), torch.tensor([slot], dtype=torch.int32, device=dev),
                            token_seq=torch.tensor([seq], dtype=torch.int32, device=dev), q_out=out, device_status=status)
        torch.cuda.synchronize()
        fine = (seq, slot) == (0, 45)
        assert int(status) == (0 if fine else -8)
        if not fine:
            assert torch.equal(kc.cpu(), k) and torch.equal(vc.cpu(), v) and bool((out == 9.0).all())


def test_no_tokens(cuda_lib):
    art, dev = cuda_lib, "cuda"
    k, v, table = ref.paged([40], 16, 2, 64, "bf16", 1, stale=0.0)
    kc, vc = k.to(dev), v.to(dev)
    e = lambda h: torch.empty(0, h, 64, dtype=torch.bfloat16, device=dev)   # noqa: E731
    none = torch.empty(0, dtype=torch.int32, device=dev)
    art.art_rope_append(art.art_rope_init(64), e(4), e(2), e(2), kc, vc, table.to(dev), none, token_seq=none)
    torch.cuda.synchronize()
    assert torch.equal(kc.cpu(), k) and torch.equal(vc.cpu(), v)


def test_offsets_past_32_bits(cuda_lib):
    art, dev = cuda_lib, "cuda"
    page, Hkv, d = 64, 8, 128
    pages = 2 ** 31 // (page * Hkv * d) + 9
    kc = torch.empty(pages, Hkv, page, d, dtype=torch.bfloat16, device=dev)
    vc = torch.empty_like(kc)
    table = torch.tensor([[pages - 1]], dtype=torch.int32, device=dev)
    kn, vn = (torch.randn(1, Hkv, d, device=dev).to(torch.bfloat16) for _ in range(2))
    art.art_rope_append(art.art_rope_init(d), torch.zeros(1, 8, d, dtype=torch.bfloat16, device=dev), kn, vn, kc, vc, table,
                        torch.tensor([63], dtype=torch.int32, device=dev),
                        positions=torch.tensor([0], dtype=torch.int32, device=dev))
    torch.cuda.synchronize()
    assert torch.equal(kc[-1, :, 63], kn[0]) and torch.equal(vc[-1, :, 63], vn[0])


@pytest.mark.parametrize("layout,d,rot", [("half", 128, 128), ("interleaved", 128, 128), ("half", 96, 90), ("half", 64, 6)])
def test_angles_to_32_bits_of_a_turn(cuda_lib, layout, d, rot):
    """Pairs (1, 0) come out as (cos, sin), with no further rounding: the angle is right to 2^-32 of a turn (below 2^-29
    rad), the sines to one and a half steps of the value (one and a half roundings of their largest terms).  Positions over all 32 bits,
    near whole, half, quarter and eighth turns too."""
    art, dev, B = cuda_lib, "cuda", 4096
    g = torch.Generator().manual_seed(rot)
    f = freqs(rot)
    pos = torch.randint(-2 ** 31, 2 ** 31, (B,), generator=g)
    pos[:1000] = torch.arange(1000)                                   # f[0] = 1: radians
    f[-1] = 2 * math.pi * 2.0 ** -12                                  # 4096 positions a turn: every eighth exactly
    pos[1000:2000] = 512 * torch.arange(1000) + torch.randint(-1, 2, (1000,), generator=g)
    x = torch.zeros(1, 1, d)
    x[..., slice(0, rot // 2) if layout == "half" else slice(0, rot, 2)] = 1.0
    x = x.to(dev).expand(B, 1, d)
    cache = torch.zeros(B, 1, 1, d, device=dev)
    out = art.art_rope_append(art.art_rope_init(d, rot_dim=rot, layout=layout, inv_freq=f), x, x, x, cache, cache.clone(),
                              torch.arange(B, dtype=torch.int32, device=dev)[:, None],
                              torch.zeros(B, dtype=torch.int32, device=dev), positions=pos.int().to(dev))
    torch.cuda.synchronize()
    first, second = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    # the angle itself needs more than 64 bits of significand: the fraction of a turn, in whole numbers
    turns = [int(t) for t in art.art_rope_init(d, rot_dim=rot, inv_freq=f).turns][:rot // 2]
    frac = np.array([[(p * t) % 2 ** 64 for t in turns] for p in pos.tolist()], dtype=np.uint64)
    eighth = ((frac + np.uint64(2 ** 60)) >> np.uint64(61)).astype(np.int64)      # so that the 64-bit sine's argument is small
    rest = (frac - (eighth.astype(np.uint64) << np.uint64(61))).view(np.int64).astype(np.float64) * (2 * math.pi / 2.0 ** 64)
    z = np.exp(1j * rest) * np.exp(2j * math.pi / 8 * eighth)
    for got, want in ((out[:, 0, first], z.real), (out[:, 0, second], z.imag)):
        got, want = got.double().cpu().numpy(), np.asarray(want)
        step = 2.0 ** (np.floor(np.log2(np.maximum(np.maximum(np.abs(got), np.abs(want)), 1e-30))) - 23)
        assert (np.abs(got - want) <= 1.5 * step + 2.0 ** -29).all(), np.abs(got - want).max()
    assert torch.equal(cache.flatten(0, 2)[:, :rot], out[:, 0, :rot])
