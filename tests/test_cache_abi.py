"""Host checks of the cache operators' entry points (no GPU): refusals come
before any CUDA call, on descriptors over never-dereferenced addresses, and
the rotary angles against high-precision arithmetic."""
import ctypes
import math
from fractions import Fraction

import pytest

from kv_cache_early_art_b200 import build
from tests.test_abi import FAKE, T

NULL, SHAPE, DTYPE, UNSUPPORTED, PARAM = -1, -2, -3, -4, -5


@pytest.fixture(scope="module")
def art():
    build.build_library()
    import kv_cache_early_art_b200 as pkg
    return pkg


def fill(p, **kw):
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def call(art, name, p):
    return getattr(art.raw_library(), name)(bytes(p), None)


# ------------------------------------------------------------------ append ----

def append_params(art, Tn=5, Hq=8, Hkv=2, d=128, page=16, NP=10, B=3, MB=4, dt=1, rot=None):
    rope = art.art_rope_init(d, rot_dim=rot)
    p = fill(art.ArtAppendParams(), q=T([Tn, Hq, d], dt), k=T([Tn, Hkv, d], dt), v=T([Tn, Hkv, d], dt),
             q_out=T([Tn, Hq, d], dt, data=FAKE + 4096), k_cache=T([NP, Hkv, page, d], dt), v_cache=T([NP, Hkv, page, d], dt),
             page_table=T([B, MB], 2), slots=T([Tn], 2), token_seq=T([Tn], 2), mass=T([B, Hkv, MB * page], 0),
             rope=ctypes.addressof(rope))
    p._rope = rope
    return p


APPEND = [
    (lambda p: setattr(p, "rope", None), NULL), (lambda p: setattr(p.q, "data", None), NULL),
    (lambda p: setattr(p.v_cache, "data", None), NULL), (lambda p: setattr(p.slots, "data", None), NULL),
    (lambda p: setattr(p.q, "ndim", 2), SHAPE), (lambda p: p.k.shape.__setitem__(0, 4), SHAPE),
    (lambda p: p.q_out.shape.__setitem__(1, 4), SHAPE), (lambda p: p.k_cache.shape.__setitem__(1, 3), SHAPE),
    (lambda p: p.v_cache.shape.__setitem__(0, 9), SHAPE), (lambda p: p.slots.shape.__setitem__(0, 6), SHAPE),
    (lambda p: p.token_seq.shape.__setitem__(0, 6), SHAPE), (lambda p: setattr(p.token_seq, "data", None), SHAPE),  # T != B
    (lambda p: p.mass.shape.__setitem__(2, 63), SHAPE), (lambda p: p.mass.stride.__setitem__(1, 0), SHAPE),
    (lambda p: p.q_out.stride.__setitem__(1, 64), SHAPE),                    # written rows overlap
    (lambda p: p.q.stride.__setitem__(2, 2), SHAPE), (lambda p: setattr(p.k_cache, "data", FAKE + 8), SHAPE),
    (lambda p: p.v_cache.stride.__setitem__(1, 4), SHAPE), (lambda p: setattr(p.slots, "data", FAKE + 2), SHAPE),
    (lambda p: setattr(p, "device_status", FAKE + 1), SHAPE),
    (lambda p: (setattr(p.q_out, "data", FAKE), p.q_out.stride.__setitem__(0, 2048)), SHAPE),   # q through other strides
    (lambda p: setattr(p.k, "dtype", 0), DTYPE), (lambda p: setattr(p.k_cache, "dtype", 0), DTYPE),
    (lambda p: setattr(p.slots, "dtype", 0), DTYPE), (lambda p: setattr(p.mass, "dtype", 1), DTYPE),
]


@pytest.mark.parametrize("i", range(len(APPEND)))
def test_append_refusals(art, i):
    p = append_params(art)
    APPEND[i][0](p)
    assert call(art, "art_rope_append", p) == APPEND[i][1]


def test_append_other_refusals(art):
    assert art.raw_library().art_rope_append(None, None) == NULL
    p = append_params(art)
    other = art.art_rope_init(64)
    p.rope = ctypes.addressof(other)
    assert call(art, "art_rope_append", p) == SHAPE                          # angles of another head size
    p = append_params(art)
    p._rope.rot_dim = 130
    assert call(art, "art_rope_append", p) == PARAM
    p = append_params(art, page=5000)
    assert call(art, "art_rope_append", p) == SHAPE
    p = append_params(art, Tn=0)
    assert call(art, "art_rope_append", p) == 0                              # nothing to do, nothing launched


def test_rope_init_refusals(art):
    ok = dict(head_dim=128)
    for kw, code in ((dict(head_dim=120), UNSUPPORTED), (dict(head_dim=272), UNSUPPORTED), (dict(head_dim=0), UNSUPPORTED),
                     (dict(rot_dim=130), PARAM), (dict(rot_dim=7), PARAM), (dict(rot_dim=-2), PARAM), (dict(base=1.0), PARAM),
                     (dict(base=math.nan), PARAM), (dict(base=math.inf), PARAM), (dict(amplitude=math.inf), PARAM),
                     (dict(scaling="linear", factor=0.0), PARAM), (dict(scaling="ntk", factor=math.nan), PARAM),
                     (dict(scaling="by_parts", factor=2.0), PARAM),
                     (dict(scaling="by_parts", factor=2.0, original_len=100, low_turns=4.0, high_turns=4.0), PARAM),
                     (dict(rot_dim=4, inv_freq=[1.0, math.inf]), PARAM)):
        with pytest.raises(art.ArtError) as e:
            art.art_rope_init(**{**ok, **kw})
        assert e.value.status == code, kw
    for kw in (dict(layout="odd"), dict(scaling="odd"), dict(inv_freq=[1.0])):
        with pytest.raises(ValueError):
            art.art_rope_init(128, **kw)
    assert art.raw_library().art_rope_init(None, 64, 64, 0, 1e4, 0, 1.0, 0, 0.0, 0.0, 1.0) == NULL


def test_rope_fractions_of_a_turn(art):
    """turns[i] = 2^64 frac(f / 2 pi) to the double's precision: against
    rational arithmetic with 2 pi to 40 digits; |error| <= 2^-53 of f / 2 pi
    for the double f itself and one half step of the long double division and
    of the rounding to 2^-64."""
    two_pi = Fraction(2 * 31415926535897932384626433832795028841971, 10 ** 40)
    freqs = [1.0, 0.5, 1e-4, 1.0 / 3.0, 2.5, -0.75, 123.456, 0.0]
    r = art.art_rope_init(16, rot_dim=16, inv_freq=freqs)
    for i, f in enumerate(freqs):
        want = Fraction(f) / two_pi % 1 * 2 ** 64
        err = abs(Fraction(r.turns[i]) - want)
        err = min(err, 2 ** 64 - err)
        assert err <= 2 ** 64 * abs(Fraction(f) / two_pi) * Fraction(1, 2 ** 62) + 3


# ------------------------------------------------------------------- split ----

def split_params(art, B=2, Hq=8, Hkv=2, d=128, page=16, NP=10, MB=500, dt=1, mass=True):
    return fill(art.ArtSplitParams(), q=T([B, Hq, d], dt), k_cache=T([NP, Hkv, page, d], dt), v_cache=T([NP, Hkv, page, d], dt),
                page_table=T([B, MB], 2), seq_lens=T([B], 2), out=T([B, Hq, d], 0, data=FAKE + (1 << 20)), lse=T([B, Hq], 0),
                mass=T([B, Hkv, MB * page], 0) if mass else art.ArtTensor(), workspace=FAKE, workspace_bytes=1 << 40)


SPLIT = [
    (lambda p: setattr(p.q, "data", None), NULL), (lambda p: setattr(p.out, "data", None), NULL),
    (lambda p: setattr(p, "workspace", None), NULL), (lambda p: setattr(p, "workspace", FAKE + 128), SHAPE),
    (lambda p: setattr(p, "workspace_bytes", 1000), SHAPE), (lambda p: setattr(p.lse, "ndim", 3), SHAPE),
    (lambda p: p.out.shape.__setitem__(2, 64), SHAPE), (lambda p: p.lse.shape.__setitem__(1, 7), SHAPE),
    (lambda p: p.mass.shape.__setitem__(2, 7999), SHAPE), (lambda p: p.mass.stride.__setitem__(0, 10), SHAPE),
    (lambda p: p.seq_lens.shape.__setitem__(0, 3), SHAPE), (lambda p: p.q.stride.__setitem__(1, 129), SHAPE),
    (lambda p: p.q.shape.__setitem__(1, 9), SHAPE), (lambda p: p.v_cache.shape.__setitem__(2, 32), SHAPE),
    (lambda p: p.k_cache.stride.__setitem__(2, 0), SHAPE), (lambda p: p.out.stride.__setitem__(0, 8), SHAPE),
    (lambda p: p.lse.stride.__setitem__(1, 0), SHAPE), (lambda p: setattr(p.k_cache, "data", FAKE + 4), SHAPE),
    (lambda p: setattr(p.v_cache, "dtype", 0), DTYPE), (lambda p: setattr(p.out, "dtype", 2), DTYPE),
    (lambda p: setattr(p.mass, "dtype", 1), DTYPE), (lambda p: setattr(p.page_table, "dtype", 1), DTYPE),
    (lambda p: setattr(p, "sm_scale", math.nan), PARAM), (lambda p: setattr(p, "sm_scale", math.inf), PARAM),
    (lambda p: setattr(p.out, "data", FAKE), PARAM),                        # q itself
]


@pytest.mark.parametrize("i", range(len(SPLIT)))
def test_split_refusals(art, i):
    p = split_params(art)
    SPLIT[i][0](p)
    assert call(art, "art_decode_attention_split", p) == SPLIT[i][1]


def test_split_sizes(art):
    lib = art.raw_library()
    assert lib.art_decode_attention_split(None, None) == NULL and lib.art_split_workspace_bytes(None) == NULL
    for kw in (dict(d=96), dict(d=32), dict(Hq=18, Hkv=2)):
        assert call(art, "art_decode_attention_split", split_params(art, **kw)) == UNSUPPORTED
        assert lib.art_split_workspace_bytes(bytes(split_params(art, **kw))) == UNSUPPORTED
    assert call(art, "art_decode_attention_split", split_params(art, page=4097)) == SHAPE
    # the workspace goes by the shapes: logits only with mass
    small, big = (lib.art_split_workspace_bytes(bytes(split_params(art, mass=m))) for m in (False, True))
    assert 0 < small < big and big - small >= 2 * 8 * 8000 * 4
    for m in (False, True):                                   # short sequences: one kernel, no workspace
        assert lib.art_split_workspace_bytes(bytes(split_params(art, mass=m, MB=64))) == 0
    p = split_params(art)
    p.workspace_bytes = big - 1
    assert call(art, "art_decode_attention_split", p) == SHAPE


# ------------------------------------------------------------------- evict ----

def evict_params(art, B=2, Hkv=2, d=128, page=16, NP=20, MB=5, NB=2, dt=1, budget=32, sink=2, recent=5, moved=True):
    p = fill(art.ArtEvictParams(), k_cache=T([NP, Hkv, page, d], dt), v_cache=T([NP, Hkv, page, d], dt),
             page_table=T([B, MB], 2), seq_lens=T([B], 2), mass=T([B, Hkv, MB * page], 0),
             new_seq_lens=T([B], 2, data=FAKE + 4096), kept=T([B, Hkv, max(budget, 1)], 2), budget=budget, sink=sink,
             recent=recent)
    if moved:
        p.new_page_table = T([B, NB], 2, data=FAKE + 8192)
        p.new_mass = T([B, Hkv, NB * page], 0, data=FAKE + 65536)
    return p


EVICT = [
    (lambda p: setattr(p.mass, "data", None), NULL), (lambda p: setattr(p.kept, "data", None), NULL),
    (lambda p: setattr(p.new_seq_lens, "data", None), NULL), (lambda p: setattr(p.mass, "ndim", 2), SHAPE),
    (lambda p: p.kept.shape.__setitem__(2, 31), SHAPE), (lambda p: p.new_page_table.shape.__setitem__(1, 1), SHAPE),
    (lambda p: p.new_mass.shape.__setitem__(2, 31), SHAPE), (lambda p: p.mass.shape.__setitem__(2, 79), SHAPE),
    (lambda p: p.kept.stride.__setitem__(1, 0), SHAPE), (lambda p: p.k_cache.stride.__setitem__(0, 3), SHAPE),
    (lambda p: p.new_seq_lens.shape.__setitem__(0, 3), SHAPE), (lambda p: setattr(p.v_cache, "dtype", 0), DTYPE),
    (lambda p: setattr(p.new_mass, "dtype", 1), DTYPE), (lambda p: setattr(p.kept, "dtype", 0), DTYPE),
    (lambda p: setattr(p, "budget", 0), PARAM), (lambda p: setattr(p, "sink", -1), PARAM),
    (lambda p: setattr(p, "recent", 31), PARAM), (lambda p: setattr(p, "recent", 2 ** 31 - 1), PARAM),
    (lambda p: setattr(p.new_seq_lens, "data", FAKE), PARAM),                # seq_lens itself
    (lambda p: (setattr(p.new_mass, "data", FAKE), p.new_mass.stride.__setitem__(1, 64)), PARAM),
]


@pytest.mark.parametrize("i", range(len(EVICT)))
def test_evict_refusals(art, i):
    p = evict_params(art)
    EVICT[i][0](p)
    assert call(art, "art_cache_evict", p) == EVICT[i][1]


def test_evict_sizes(art):
    assert art.raw_library().art_cache_evict(None, None) == NULL
    assert call(art, "art_cache_evict", evict_params(art, d=4)) == SHAPE                   # 8-byte rows
    assert call(art, "art_cache_evict", evict_params(art, d=1032)) == UNSUPPORTED          # rows over 2048 bytes
    assert call(art, "art_cache_evict", evict_params(art, MB=393216 // 16 + 1, moved=False)) == UNSUPPORTED


# ----------------------------------------------------------------- binding ----

def test_bindings_refuse_cpu_tensors(art):
    import torch
    z = torch.zeros
    i32 = torch.int32
    with pytest.raises(ValueError):
        art.art_rope_append(art.art_rope_init(64), z(1, 4, 64), z(1, 2, 64), z(1, 2, 64), z(9, 2, 16, 64), z(9, 2, 16, 64),
                            z(1, 2, dtype=i32), z(1, dtype=i32))
    with pytest.raises(ValueError):
        art.art_decode_attention_split(z(1, 4, 64), z(9, 2, 16, 64), z(9, 2, 16, 64), z(1, 2, dtype=i32), z(1, dtype=i32))
    with pytest.raises(ValueError):
        art.art_cache_evict(z(9, 2, 16, 64), z(9, 2, 16, 64), z(1, 2, dtype=i32), z(1, dtype=i32), z(1, 2, 32), 8)


def test_structures_match_the_header(art):
    """Sizes and the last fields' places of the C structures, compiled from art.h."""
    import os
    import subprocess
    import tempfile
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = ('#include <stdio.h>\n#include <stddef.h>\n#include "art.h"\nint main(void){printf("%zu %zu %zu %zu %zu %zu %zu %zu",'
           'sizeof(art_append_params_t),offsetof(art_append_params_t,device_status),sizeof(art_split_params_t),'
           'offsetof(art_split_params_t,workspace_bytes),sizeof(art_evict_params_t),offsetof(art_evict_params_t,device_status),'
           'sizeof(art_rope_t),offsetof(art_rope_t,turns));return 0;}')
    with tempfile.TemporaryDirectory() as d:
        open(os.path.join(d, "a.c"), "w").write(src)
        subprocess.check_call(["gcc", "-I", os.path.join(root, "include"), "-o", os.path.join(d, "a"), os.path.join(d, "a.c")])
        got = [int(x) for x in subprocess.check_output([os.path.join(d, "a")]).split()]
    S = ctypes.sizeof
    assert got == [S(art.ArtAppendParams), art.ArtAppendParams.device_status.offset, S(art.ArtSplitParams),
                   art.ArtSplitParams.workspace_bytes.offset, S(art.ArtEvictParams), art.ArtEvictParams.device_status.offset,
                   S(art.ArtRope), art.ArtRope.turns.offset]


def test_workspace_query_needs_no_out(art):
    """Its size goes by the inputs: without an out, and for queries broadcast over the batch or the heads."""
    query = art.raw_library().art_split_workspace_bytes
    want = query(bytes(split_params(art)))
    p = split_params(art)
    p.out = art.ArtTensor()
    assert want > 0 and query(bytes(p)) == want
    for i in (0, 1):
        p.q.stride[i] = 0
        assert query(bytes(p)) == want
    p = split_params(art)
    p.out.shape[2] = 64
    assert query(bytes(p)) == SHAPE                                          # one that is given is checked


def test_empty_tensors_are_no_absent_arguments(art):
    """Data and no elements: the shape checks refuse them (the binding passes a tensor of no elements like this)."""
    def empty(t, axis):
        t.shape[axis] = 0
        return t
    p = evict_params(art)
    empty(p.new_page_table, 1)
    assert call(art, "art_cache_evict", p) == SHAPE
    p = evict_params(art)
    empty(p.new_mass, 2)
    assert call(art, "art_cache_evict", p) == SHAPE
    for name, axis in (("positions", 0), ("token_seq", 0), ("mass", 2)):
        p = append_params(art, Tn=3)                                         # as many tokens as sequences
        p.positions = T([3], 2)
        empty(getattr(p, name), axis)
        assert call(art, "art_rope_append", p) == SHAPE, name
    for name in ("lse", "mass"):
        p = split_params(art)
        empty(getattr(p, name), 1)
        assert call(art, "art_decode_attention_split", p) == SHAPE, name
    p = append_params(art, Tn=0)
    p.positions = T([0], 2)
    assert call(art, "art_rope_append", p) == 0                              # no tokens, so no positions


def test_workspace_must_hold_the_bytes_it_counts(art):
    """An expanded or strided workspace has fewer bytes behind its address than elements: refused before anything runs."""
    import torch
    z, i32 = torch.zeros, torch.int32
    args = (z(1, 4, 64), z(9, 2, 16, 64), z(9, 2, 16, 64), z(1, 2, dtype=i32), z(1, dtype=i32))
    for ws in (z(1, dtype=torch.uint8).expand(1 << 24), z(4096)[::2], z(64, 64).t()):
        with pytest.raises(ValueError, match="contiguous"):
            art.art_decode_attention_split(*args, workspace=ws)


def test_factors_that_leave_the_floats_are_refused(art):
    """Finite where they are given, infinite where they are used."""
    for amplitude, ok in ((1e300, False), (-1e39, False), (3e38, True)):
        if ok:
            assert art.art_rope_init(64, amplitude=amplitude).amplitude > 2.9e38
        else:
            with pytest.raises(art.ArtError) as e:
                art.art_rope_init(64, amplitude=amplitude)
            assert e.value.status == PARAM
    query = art.raw_library().art_split_workspace_bytes
    for scale, ok in ((3e38, False), (2.4e38, False), (2.3e38, True), (-1.0, True)):
        p = split_params(art)
        p.sm_scale = scale
        assert (query(bytes(p)) > 0) == ok
        if not ok:
            assert call(art, "art_decode_attention_split", p) == PARAM


def test_written_tensors_hold_no_element_twice(art):
    """Two dimensions that each clear a row but not one another, or equal strides; permuted and padded ones pass."""
    def attend(**strides):
        p = split_params(art)
        for name, s in strides.items():
            for i, x in enumerate(s):
                getattr(p, name).stride[i] = x
        return art.raw_library().art_split_workspace_bytes(bytes(p))
    for bad in (dict(lse=(1, 1)), dict(lse=(2, 1)), dict(lse=(8, 0)), dict(lse=(7, 1)), dict(out=(128, 128, 1)),
                dict(out=(128 * 7, 128, 1)), dict(mass=(8000, 8000, 1)), dict(mass=(8000, 12000, 1))):
        assert attend(**bad) == SHAPE, bad
    for good in (dict(lse=(8, 1)), dict(lse=(1, 2)), dict(lse=(32, 4)), dict(out=(128, 256, 1)), dict(out=(1200, 130, 1)),
                 dict(mass=(8000, 16000, 1)), dict(mass=(2 ** 62, 8000, 1))):
        assert attend(**good) > 0, good

    def refused(p, name, tensor, strides):
        for i, x in enumerate(strides):
            getattr(p, tensor).stride[i] = x
        return call(art, name, p) == SHAPE
    assert refused(append_params(art), "art_rope_append", "q_out", (128, 128, 1))
    assert refused(append_params(art), "art_rope_append", "q_out", (512, 128, 1))
    assert refused(append_params(art), "art_rope_append", "mass", (64, 64, 1))
    assert refused(append_params(art), "art_rope_append", "v_cache", (2048, 2048, 128, 1))
    assert refused(evict_params(art), "art_cache_evict", "kept", (32, 32, 1))
    assert refused(evict_params(art), "art_cache_evict", "new_mass", (40, 32, 1))
    assert refused(evict_params(art), "art_cache_evict", "k_cache", (4096, 2048, 64, 1))
    # masses that are only read, to become new_mass, may overlap (the query makes the call's checks)
    p = evict_params(art)
    p.mass.stride[0] = p.mass.stride[1] = 80
    assert art.raw_library().art_evict_cluster_size(bytes(p)) > 0
    p.new_mass = art.ArtTensor()                                             # in place they are written
    assert art.raw_library().art_evict_cluster_size(bytes(p)) == SHAPE


def test_evict_cluster_size(art):
    """The query makes the call's checks; a short unit takes one CTA, the longest table eight."""
    query = art.raw_library().art_evict_cluster_size
    assert query(None) == NULL
    for change, code in EVICT:
        p = evict_params(art)
        change(p)
        assert query(bytes(p)) == code
    assert query(bytes(evict_params(art))) == 1
    assert query(bytes(evict_params(art, MB=393216 // 16, moved=False))) == 8


@pytest.mark.parametrize("dt,d,Hq,tile", [(1, 128, 32, 16), (1, 256, 32, 16), (0, 64, 32, 16), (0, 128, 32, 8), (0, 128, 40, 16),
                                          (0, 256, 8, 8), (0, 256, 64, 8)])
def test_most_tokens_of_an_attention(art, dt, d, Hq, tile):
    """Tiles of all units below 2^31: 2^15 units here, so tables of less than 2^16 tiles each."""
    query = art.raw_library().art_split_workspace_bytes
    fits = dict(B=4096, Hkv=8, Hq=Hq, d=d, dt=dt, page=tile, mass=False)
    assert query(bytes(split_params(art, MB=65535, **fits))) > 0
    assert query(bytes(split_params(art, MB=65536, **fits))) == UNSUPPORTED
