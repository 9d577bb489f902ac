"""GPU tests of art_decode_attention_split against its 64-bit definition.

Error bounds (tests/cache_ref.py derives the logit's and the weight's): an
output is a sum of n weighted values, accumulated in fp32 over at most n / 16
+ 64 steps of 2^-23, with weights used twice (numerator and sum) and, on the
bf16 path, as three bf16 terms (each rounding at most half a step, 2^-8 of what
is left: 2^-24)."""
import math

import pytest
import torch

from tests import cache_ref as ref

pytestmark = pytest.mark.gpu


def check(art, q, k, v, table, lens, *, mass0=None, out=None, lse=None, **kw):
    """Runs the call on GPU copies and checks out, lse and mass."""
    B, Hq, d = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    dev = "cuda"
    mass = None if mass0 is None else mass0.to(dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    sl = torch.tensor(lens, dtype=torch.int32, device=dev)
    o, e = art.art_decode_attention_split(q.to(dev), k.to(dev), v.to(dev), table.to(dev), sl, mass=mass, out=out,
                                          lse=lse, device_status=status, **kw)
    torch.cuda.synchronize()
    assert int(status) == 0
    verify(q, k, v, table, lens, o, e, mass0, mass, kw.get("sm_scale"))
    return o, e


def verify(q, k, v, table, lens, o, e, mass0=None, mass=None, scale=None):
    B, Hq, d = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    want, lse64, weights, size, top, spread = ref.attend(q, k, v, table, lens, scale)
    n = torch.tensor([max(0, int(x)) for x in lens], dtype=torch.float64)[:, None]
    werr = ref.weight_error(d, n, size, top, lse64)
    tol = (2 * (werr + 2.0 ** -24)[..., None] + (n[..., None] / 16 + 64) * 2.0 ** -23) * spread
    if o.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * want.abs()
    err = (o.double().cpu() - want).abs()
    assert bool((err <= tol).all()), f"output off by {float((err / tol.clamp(min=1e-300)).max()):.2f} of its bound"
    e = e.double().cpu()
    empty = torch.isinf(lse64)
    assert bool((e[empty] == -math.inf).all()) and bool((o.double().cpu()[empty] == 0).all())
    lerr = ref.logit_error(d, size, top, lse64) + n * 2.0 ** -24 + 2.0 ** -20
    assert bool(((e - lse64).abs()[~empty] <= lerr.expand_as(e)[~empty]).all())
    if mass0 is None:
        return
    got = mass.double().cpu()
    for b in range(B):
        m = max(0, int(lens[b]))
        old = mass0[b].double()
        # one rounding a head and one of the sum
        rel = werr[b].view(Hkv, G).amax(-1)[:, None] + (G + 1) * 2.0 ** -24
        target = old[:, :m] + weights[b]
        tol = rel * weights[b] + 2.0 ** -24 * target.abs()
        assert bool(((got[b, :, :m] - target).abs() <= tol).all())
        assert torch.equal(got[b, :, m:], old[:, m:])        # columns of no token stay


def make(lens, Hq, Hkv, d, page, dtype, seed, gain=2.0, **kw):
    k, v, table = ref.paged(lens, page, Hkv, d, dtype, seed, **kw)
    g = torch.Generator().manual_seed(seed + 1000)
    q = (gain * torch.randn(len(lens), Hq, d, generator=g)).to(ref.DT[dtype])
    return q, k, v, table


def random_mass(table, k, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.rand(table.shape[0], k.shape[1], table.shape[1] * k.shape[2], generator=g)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 3, 4, 5, 8])
def test_heads_and_types(cuda_lib, dtype, d, G):
    lens = [1, 15, 16, 17, 0, 333, 1025]
    q, k, v, table = make(lens, 2 * G, 2, d, 16, dtype, seed=G + d)
    check(cuda_lib, q, k, v, table, lens, mass0=random_mass(table, k))


@pytest.mark.parametrize("page", [1, 5, 16, 24, 64, 300])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_page_sizes(cuda_lib, page, dtype):
    """Pages that end inside a tile, of one row, and longer than a sequence."""
    lens = [700, 1, 299, 301, 2 * page, 2 * page + 1]
    q, k, v, table = make(lens, 12, 3, 64, page, dtype, seed=page)
    check(cuda_lib, q, k, v, table, lens, mass0=random_mass(table, k))


@pytest.mark.parametrize("width", [8, 9, 16, 17, 32, 33, 64, 65])
@pytest.mark.parametrize("dtype,d,G", [("bf16", 128, 4), ("bf16", 256, 8), ("f32", 64, 1), ("f32", 256, 5), ("bf16", 64, 7)])
def test_clusters(cuda_lib, width, dtype, d, G):
    """Tables on both sides of each number of CTAs on a unit, and past the longest; sequences that leave CTAs without a tile."""
    lens = [16 * width, 16 * width - 1, 1, 0, 100]
    lens = [min(n, 16 * width) for n in lens]
    q, k, v, table = make(lens, 2 * G, 2, d, 16, dtype, seed=width)
    check(cuda_lib, q, k, v, table, lens, mass0=random_mass(table, k))


@pytest.mark.parametrize("L", [300, 3000])
def test_without_lse(cuda_lib, L):
    """The C entry point takes no lse, in either kernel."""
    from kv_cache_early_art_b200 import binding
    q, k, v, table = make([L], 4, 2, 64, 16, "bf16", seed=L)
    g = [x.cuda() for x in (q, k, v, table)] + [torch.tensor([L], dtype=torch.int32, device="cuda")]
    o, e = cuda_lib.art_decode_attention_split(*g)
    o2 = torch.empty_like(o)
    ws = torch.empty(max(1, cuda_lib.art_split_workspace_bytes(*g)), dtype=torch.uint8, device="cuda")
    binding._run("art_decode_attention_split", None, (*g, o2, None, None), (ws,),
                 binding._SPLIT_TAIL.pack(0.0, 0, 0, ws.data_ptr(), ws.numel()))
    torch.cuda.synchronize()
    assert torch.equal(o, o2)


@pytest.mark.parametrize("lens", [[1], [8200], [0, 0, 0], [0, 5, 0, 0, 3, 0], [4097, 1, 1, 1, 1, 1], [-4, 7]])
@pytest.mark.parametrize("mass", [False, True])
def test_lengths(cuda_lib, lens, mass):
    q, k, v, table = make(lens, 8, 2, 128, 64, "bf16", seed=len(lens))
    check(cuda_lib, q, k, v, table, lens, mass0=random_mass(table, k) if mass else None)


def test_many_short_sequences(cuda_lib):
    """More units than CTAs, each a few tiles, some empty: shares that hold many whole units."""
    lens = [(i * 37) % 90 for i in range(600)]
    q, k, v, table = make(lens, 4, 2, 64, 16, "bf16", seed=3)
    check(cuda_lib, q, k, v, table, lens, mass0=random_mass(table, k))


def test_long_unit_over_all_ctas(cuda_lib):
    """One unit, joined from every CTA's part."""
    q, k, v, table = make([40000], 7, 1, 128, 64, "bf16", seed=4)
    check(cuda_lib, q, k, v, table, [40000], mass0=random_mass(table, k))


def test_table_wider_than_the_sequences(cuda_lib):
    lens = [100, 513]
    q, k, v, table = make(lens, 8, 2, 128, 64, "bf16", seed=5, width=400)
    check(cuda_lib, q, k, v, table, lens, mass0=random_mass(table, k))


@pytest.mark.parametrize("stale", [math.inf, -math.inf])
def test_stale_rows_may_hold_anything(cuda_lib, stale):
    lens = [37, 130]
    q, k, v, table = make(lens, 8, 2, 128, 64, "bf16", seed=6, stale=stale)
    check(cuda_lib, q, k, v, table, lens)
    q, k, v, table = make(lens, 4, 2, 64, 24, "f32", seed=6, stale=stale)
    check(cuda_lib, q, k, v, table, lens)


def test_sharp_and_flat_logits(cuda_lib):
    """One token with nearly all the weight, first, last and in the middle; and all equal."""
    lens = [1000] * 4
    q, k, v, table = make(lens, 4, 1, 128, 64, "bf16", seed=7)
    for b, t in ((0, 0), (1, 500), (2, 999)):
        k[table[b, t // 64].long(), 0, t % 64] = (q[b, 0].float() * 2).to(torch.bfloat16)
    q[3] = 0
    check(cuda_lib, q, k, v, table, lens, mass0=random_mass(table, k))


def test_scale_and_bf16_output(cuda_lib):
    lens = [513, 64]
    q, k, v, table = make(lens, 8, 2, 128, 64, "bf16", seed=8)
    o = torch.empty(2, 8, 128, dtype=torch.bfloat16, device="cuda")
    check(cuda_lib, q, k, v, table, lens, sm_scale=0.05, out=o)


def test_strided_tensors(cuda_lib):
    """Cache with the heads inside the rows, v laid out otherwise, padded q, out, lse, table and mass."""
    lens = [333, 100]
    q, k, v, table = make(lens, 6, 2, 64, 16, "bf16", seed=9)
    kk = torch.empty(k.shape[0], 16, 2, 64 + 8, dtype=k.dtype).permute(0, 2, 1, 3)[..., :64]
    kk.copy_(k)
    vv = torch.empty(v.shape[0], 3, 16, 64, dtype=v.dtype)[:, 1:]
    vv.copy_(v)
    qq = torch.empty(2, 7, 96, dtype=q.dtype)[:, 1:, 8:72]
    qq.copy_(q)
    dev = "cuda"
    tt = torch.full((2, table.shape[1] + 3), -7, dtype=torch.int32)
    tt[:, :table.shape[1]] = table
    tt = tt.to(dev)[:, :table.shape[1]]
    # .to() keeps the strides of a dense permutation only, so move the bases
    kg = torch.empty(k.shape[0], 16, 2, 72, dtype=k.dtype, device=dev).permute(0, 2, 1, 3)[..., :64]
    kg.copy_(kk)
    vg = torch.empty(v.shape[0], 3, 16, 64, dtype=v.dtype, device=dev)[:, 1:]
    vg.copy_(vv)
    qg = torch.empty(2, 7, 96, dtype=q.dtype, device=dev)[:, 1:, 8:72]
    qg.copy_(qq)
    o = torch.full((2, 8, 65), 5.0, device=dev)
    e = torch.full((2, 6, 2), 5.0, device=dev)
    m0 = random_mass(table, k)
    mg = torch.full((2, 3, m0.shape[2] + 5), 5.0, device=dev)
    mg[:, :2, :m0.shape[2]] = m0.to(dev)
    sl = torch.tensor(lens, dtype=torch.int32, device=dev)
    cuda_lib.art_decode_attention_split(qg, kg, vg, tt, sl, out=o[:, 1:7, :64], lse=e[..., 0],
                                        mass=mg[:, :2, :m0.shape[2]])
    torch.cuda.synchronize()
    verify(q, k, v, table, lens, o[:, 1:7, :64], e[..., 0], m0, mg[:, :2, :m0.shape[2]])
    for edge in (o[:, 0], o[:, 7], o[:, 1:7, 64], e[..., 1], mg[:, 2], mg[:, :2, m0.shape[2]:]):
        assert bool((edge == 5.0).all())


def test_offsets_past_32_bits(cuda_lib):
    """Pages whose element offsets exceed 2^31 (the cache serves as K and as V)."""
    page, Hkv, d = 64, 8, 128
    pages = 2 ** 31 // (page * Hkv * d) + 40
    cache = torch.empty(pages, Hkv, page, d, dtype=torch.bfloat16, device="cuda")
    used = [pages - 1, 3, pages - 20]
    table = torch.tensor([used], dtype=torch.int32)
    small, _, _ = ref.paged([3 * page], page, Hkv, d, "bf16", seed=10, spare=0)
    cache[torch.tensor(used)] = small.cuda()
    q = torch.randn(1, 16, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    sl = torch.tensor([150], dtype=torch.int32, device="cuda")
    o, e = cuda_lib.art_decode_attention_split(q.cuda(), cache, cache, table.cuda(), sl)
    torch.cuda.synchronize()
    verify(q, small, small, torch.tensor([[0, 1, 2]], dtype=torch.int32), [150], o, e)


def test_bad_pages_and_long_sequences_are_reported(cuda_lib):
    lens = [200, 130]
    q, k, v, table = make(lens, 8, 2, 128, 64, "bf16", seed=11)
    dev = "cuda"
    bad = table.clone()
    bad[0, 1] = k.shape[0]
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    sl = torch.tensor(lens, dtype=torch.int32, device=dev)
    mass = random_mass(table, k).to(dev)
    m0 = mass.clone()
    o, e = cuda_lib.art_decode_attention_split(q.to(dev), k.to(dev), v.to(dev), bad.to(dev), sl, mass=mass,
                                               device_status=status)
    torch.cuda.synchronize()
    assert int(status) == -8
    # sequence 0 without its page 1, sequence 1 untouched
    t2 = table.clone()
    t2[0, 1:3] = table[0, 2:4]
    verify(q, k, v, t2, [136, 130], o, e)
    assert torch.equal(mass[0, :, 64:128], m0[0, :, 64:128])
    status.zero_()
    o, e = cuda_lib.art_decode_attention_split(q.to(dev), k.to(dev), v.to(dev), table.to(dev)[:, :2], sl,
                                               device_status=status)
    torch.cuda.synchronize()
    assert int(status) == -8
    verify(q, k, v, table, [128, 128], o, e)


def test_other_stream_and_captured_graphs_sharing_a_workspace(cuda_lib):
    """Two captured calls use one workspace in turn; replays follow new inputs."""
    dev = "cuda"
    calls = []
    for seed, lens in ((12, [900, 37]), (13, [5, 2000])):
        q, k, v, table = make(lens, 8, 2, 128, 64, "bf16", seed=seed)
        g = [x.to(dev) for x in (q, k, v, table)] + [torch.tensor(lens, dtype=torch.int32, device=dev)]
        calls.append(((q, k, v, table, lens), g, random_mass(table, k)))
    need = max(cuda_lib.art_split_workspace_bytes(*g, mass=m.to(dev)) for _, g, m in calls)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=dev)
    side = torch.cuda.Stream()
    graphs = []
    for _, g, m in calls:
        mass = m.to(dev)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            o, e = cuda_lib.art_decode_attention_split(*g, mass=mass, workspace=ws)
        side.synchronize()
        mass.copy_(m)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            cuda_lib.art_decode_attention_split(*g, mass=mass, workspace=ws, out=o, lse=e)
        graphs.append((gr, o, e, mass))
    for _ in range(2):
        for (_, g, m), (gr, o, e, mass) in zip(calls, graphs):
            mass.copy_(m)
            o.zero_()
            gr.replay()
        torch.cuda.synchronize()
        for (c, g, m), (gr, o, e, mass) in zip(calls, graphs):
            verify(*c, o, e, m, mass)
    # the captured call reads its inputs at replay
    (c, g, m), (gr, o, e, mass) = calls[0], graphs[0]
    g[0].mul_(0.5)
    mass.copy_(m)
    gr.replay()
    torch.cuda.synchronize()
    verify(c[0] * 0.5, *c[1:], o, e, m, mass)


def test_equal_inputs_give_equal_bits(cuda_lib):
    lens = [3000, 17, 801]
    q, k, v, table = make(lens, 28, 4, 128, 64, "bf16", seed=14)
    m0 = random_mass(table, k)
    runs = []
    for i in range(3):
        mass = m0.cuda()
        o, e = cuda_lib.art_decode_attention_split(q.cuda(), k.cuda(), v.cuda(), table.cuda(),
                                                   torch.tensor(lens, dtype=torch.int32).cuda(), mass=mass)
        runs.append((o, e, mass))
    for r in runs[1:]:
        assert all(torch.equal(x, y) for x, y in zip(runs[0], r))


def test_agrees_with_the_walk_at_zero_thresholds(cuda_lib):
    """art_decode_attention with both thresholds 0 is the same attention: each is within its own bound of it."""
    lens = [1000, 64, 4096]
    q, k, v, table = make(lens, 8, 2, 128, 64, "bf16", seed=15, stale=0.0)
    g = [x.cuda() for x in (q, k, v, table)]
    sl = torch.tensor(lens, dtype=torch.int32).cuda()
    walk, _ = cuda_lib.art_decode_attention(*g, None, sl, 0.0, 0.0, 1, 1)
    o, e = cuda_lib.art_decode_attention_split(*g, sl)
    torch.cuda.synchronize()
    verify(q, k, v, table, lens, o, e)
    assert float((walk - o).abs().max()) < 2e-3              # the walk's documented bf16 tolerance


@pytest.mark.parametrize("L", [300, 3000])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_broadcast_queries(cuda_lib, L, dtype):
    """One query expanded over the batch, over the heads, or both (strides of 0), with and without a given workspace."""
    lens = [L, L // 2]
    q, k, v, table = make(lens, 8, 2, 128, 64, dtype, seed=L)
    dev = "cuda"
    g = [x.to(dev) for x in (k, v, table)] + [torch.tensor(lens, dtype=torch.int32, device=dev)]
    for x in (q[:1], q[:, :1], q[:1, :1]):
        full, xg = x.expand(2, 8, 128), x.to(dev).expand(2, 8, 128)
        need = cuda_lib.art_split_workspace_bytes(xg, *g)
        ws = torch.empty(max(1, need), dtype=torch.uint8, device=dev)
        for given in (None, ws):
            o, e = cuda_lib.art_decode_attention_split(xg, *g, workspace=given)
            torch.cuda.synchronize()
            verify(full, k, v, table, lens, o, e)


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("L", [90, 3000])
@pytest.mark.parametrize("dtype,d,G", [("bf16", 128, 4), ("bf16", 64, 8), ("f32", 128, 3), ("f32", 256, 8)])
def test_logits_past_what_a_float_resolves(cuda_lib, sign, L, dtype, d, G):
    """Logits around 2^33 (and all below -2^33): products of one channel, exact in fp32, steps of 2^20 and more apart.
    The largest token's weight is 1, however far its logit in base 2 is from a float, and all others' are 0, so outputs
    and masses are copies; the log-sum-exp is that logit, rounded in the scale, its product and the change of base (half a
    step each)."""
    dev, heads = "cuda", 2
    lens = [L, L // 2 + 1, 1]
    q, k, v, table = make(lens, heads * G, heads, d, 16, dtype, seed=L + d)
    q.zero_()
    q[..., 0] = 2.0 ** 16 * torch.tensor([1.0 + i / 64 for i in range(heads * G)]).to(q.dtype)
    k.zero_()
    best = torch.zeros(len(lens), heads, dtype=torch.long)
    g = torch.Generator().manual_seed(L)
    for b, n in enumerate(lens):
        for h in range(heads):
            t = torch.arange(n)
            rank = torch.randperm(n, generator=g)                    # 0: the largest
            size = torch.where(rank == 0, 2.0 ** 17 * (1 + h / 8 + b / 16), 2.0 ** 15 * (1 + rank % 100 / 128))
            size = size if sign > 0 else -(2.0 ** 17 * (1 + (rank > 0) * (0.5 + rank % 10 / 32) + h / 16))
            k[table[b, t // 16].long(), h, t % 16, 0] = size.to(k.dtype)
            best[b, h] = int((rank == 0).nonzero())
    m0 = random_mass(table, k)
    mass = m0.to(dev)
    o, e = cuda_lib.art_decode_attention_split(q.to(dev), k.to(dev), v.to(dev), table.to(dev),
                                               torch.tensor(lens, dtype=torch.int32, device=dev), sm_scale=1.0, mass=mass)
    torch.cuda.synchronize()
    for b, n in enumerate(lens):
        for h in range(heads):
            t = int(best[b, h])
            at = (int(table[b, t // 16]), h, t % 16)
            assert torch.equal(o[b, h * G:(h + 1) * G].cpu(), v[at].float().expand(G, d)), (b, h)
            want = q[b, h * G:(h + 1) * G, 0].double() * k[at][0].double()
            assert bool(((e[b, h * G:(h + 1) * G].cpu().double() - want).abs() <= 4 * 2.0 ** -24 * want.abs()).all())
            m0[b, h, t] += G
    assert torch.equal(mass.cpu(), m0)
