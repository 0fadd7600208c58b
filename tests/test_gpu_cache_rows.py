"""Rows appended to the cache of a ragged batch, and entries read back: bit for bit as csa2_cache_write and
csa2_cache_write_projected write them and as the FP4 format defines them."""
import pytest
import torch

from test_gpu_operators import BF, F, HF, csa, decode, fp4, gen, randn  # noqa: F401

pytestmark = pytest.mark.gpu

MARK = 0xA5


def caches(csa, B, cap, d_idx, ratio):
    c = csa.Cache(B, cap, d_idx, ratio=ratio)
    for t in (c.lat_codes, c.lat_scales, c.ikey_codes, c.ikey_scales):
        t.fill_(MARK)
    return c


def planes(c):
    return c.lat_codes, c.lat_scales, c.ikey_codes, c.ikey_scales


def append_case(csa, B, R, P, pos0, cap, ratio=2, d_idx=128, keys=True, path=None, seed=0, alias=False):
    """an append against one csa2_cache_write call a sequence of the rows that its path takes"""
    g = gen(seed)
    rows = randn((B, R, 512), g, BF) * torch.exp2(randn((B, R, 1), g)).to(BF)
    prev = randn((B, 512), g, BF)
    w0, w1 = torch.rand(512, device="cuda", generator=g), torch.rand(512, device="cuda", generator=g)
    wik = fp4((d_idx, 512), g) if keys else (None, None)
    pos0 = torch.as_tensor(pos0, device="cuda", dtype=torch.int64).expand(B).contiguous()
    if path is not None:
        path = torch.as_tensor(path, device="cuda", dtype=torch.int32).expand(B, -1).contiguous()
    got, want = caches(csa, B, cap, d_idx, ratio), caches(csa, B, cap, d_idx, ratio)
    last = prev.clone()
    for b in range(B):
        steps = list(range(P)) if path is None else path[b].tolist()
        take = []
        for j in steps:
            if not 0 <= j < R:
                break
            take.append(j)
        p, r = int(pos0[b]), rows[b, take]
        if ratio == 2:
            r = torch.cat((prev[b:b + 1], r))
            last[b] = r[-1]
            p -= 1
            if p % 2:
                p, r = p + 1, r[1:]
            r = r[:len(r) // 2 * 2]
        if p < 0:
            r, p = r[-p:], 0
        n = max(0, min(len(r), cap * ratio - p))
        if n == 0:
            continue
        one = csa.Cache.of(*(t[b:b + 1] for t in planes(want)), ratio=ratio)
        r = r[None, :n].contiguous()
        if keys:
            csa.csa2_cache_write_projected(one, r, p, w0, w1, *wik)
        else:
            csa.csa2_cache_write(one, r, p, w0, w1)
    keep = prev.clone()
    out = (prev if alias else torch.zeros_like(prev)) if ratio == 2 else None
    csa.csa2_cache_append(got, rows, pos0, path=path, prev=prev if ratio == 2 else None, prev_out=out, w0=w0 if ratio == 2 else None,
                          w1=w1 if ratio == 2 else None, wik_codes=wik[0], wik_scales=wik[1])
    for a, w in zip(planes(got), planes(want)):
        assert torch.equal(a, w)
    if ratio == 2:
        assert torch.equal(out, last)
        assert alias or torch.equal(prev, keep)
    return got


@pytest.mark.parametrize("P", [1, 2, 3, 7, 8, 9, 15, 16, 17, 31, 63, 64, 65, 127, 130, 300, 1025])
@pytest.mark.parametrize("ratio", [1, 2])
@pytest.mark.parametrize("keys", [True, False])
def test_append_sizes(csa, P, ratio, keys):
    append_case(csa, 3, P, P, [0, 5, 40], 1200, ratio=ratio, keys=keys, seed=P)


@pytest.mark.parametrize("d_idx", [64, 128])
@pytest.mark.parametrize("B", [1, 2, 65, 300])
@pytest.mark.parametrize("ratio", [1, 2])
def test_append_steps_of_a_ragged_batch(csa, d_idx, B, ratio):
    pos0 = (37 * torch.arange(B)) % 211
    append_case(csa, B, 1, 1, pos0, 220, ratio=ratio, d_idx=d_idx, seed=B)
    append_case(csa, B, 5, 5, pos0, 220, ratio=ratio, d_idx=d_idx, seed=B, alias=True)


@pytest.mark.parametrize("ratio", [1, 2])
@pytest.mark.parametrize("alias", [True, False])
def test_append_paths(csa, ratio, alias):
    path = [[0, 3, 4, 9, -1, -1], [7, 7, 7, 0, 1, 15], [-1, 2, 3, 4, 5, 6], [2, -1, 3, 4, 5, 6], [15, 16, 1, 1, 1, 1],
            [1, 2, 3, -(1 << 31), 4, 5], [1, (1 << 31) - 1, 3, 4, 5, 6], [5, 6, 7, 8, -1, 9]]
    for first in (10, 11):
        append_case(csa, 8, 16, 6, [first + i for i in range(8)], 60, ratio=ratio, path=path, seed=first, alias=alias)


def test_append_long_paths(csa):
    g = gen(4)
    path = torch.randint(0, 700, (3, 2000), generator=g, device="cuda", dtype=torch.int32)
    path[0, 1999] = -1
    path[1, 257] = 700
    path[2, 256:258] = -1
    for ratio in (1, 2):
        append_case(csa, 3, 700, 2000, [3, 10, 0], 2100, ratio=ratio, path=path, keys=ratio == 1)


@pytest.mark.parametrize("ratio", [1, 2])
def test_append_at_the_edges_of_the_cache(csa, ratio):
    """positions before the cache and past it are not written"""
    big = (1 << 63) - 1
    pos0 = [-3, -20, 0, 90, 99, 100, 101, 250, big - 3, -big, 1 << 40, -(1 << 40)]
    append_case(csa, 12, 13, 13, pos0, 100 // ratio, ratio=ratio, seed=ratio)


def test_append_nothing(csa):
    for ratio in (1, 2):
        append_case(csa, 2, 4, 0, [3, 4], 20, ratio=ratio, path=torch.zeros((2, 0), dtype=torch.int32))
        append_case(csa, 2, 0, 0, [3, 4], 20, ratio=ratio)


def test_append_step_by_step_equals_one_call(csa):
    """pieces of any length one after the other, the carried row in place: the bytes of one long append"""
    g = gen(6)
    B, n = 3, 60
    rows = randn((B, n, 512), g, BF)
    w = [torch.rand(512, device="cuda", generator=g) for _ in range(2)]
    wik = fp4((128, 512), g)
    pos0 = torch.tensor([4, 7, 0], device="cuda")
    one, many = caches(csa, B, 40, 128, 2), caches(csa, B, 40, 128, 2)
    prev = randn((B, 512), g, BF)
    carried = prev.clone()
    csa.csa2_cache_append(one, rows, pos0, prev=prev, w0=w[0], w1=w[1], wik_codes=wik[0], wik_scales=wik[1])
    at = 0
    for m in [1, 1, 2, 3, 1, 5, 8, 1, 13, 25]:
        csa.csa2_cache_append(many, rows[:, at:at + m].contiguous(), pos0 + at, prev=carried, prev_out=carried, w0=w[0], w1=w[1],
                              wik_codes=wik[0], wik_scales=wik[1])
        at += m
    assert at == n and torch.equal(carried, rows[:, -1])
    for a, b in zip(planes(one), planes(many)):
        assert torch.equal(a, b)


def test_append_past_32_bit_offsets(csa):
    cap = 9_000_000                                          # 2.3 GB of codes a sequence
    g = gen(1)
    c = csa.Cache(2, cap, 64, ratio=1)
    rows = randn((2, 3, 512), g, BF)
    wik = fp4((64, 512), g)
    pos0 = torch.tensor([cap - 3, cap - 2], device="cuda")
    csa.csa2_cache_append(c, rows, pos0, wik_codes=wik[0], wik_scales=wik[1])
    small = csa.Cache(2, 8, 64, ratio=1)
    csa.csa2_cache_append(small, rows, torch.tensor([5, 6], device="cuda"), wik_codes=wik[0], wik_scales=wik[1])
    for a, b in zip(planes(c), planes(small)):
        assert torch.equal(a[:, -3:], b[:, -3:])
        assert not a[:, :cap - 3].any()
    for keys in (False, True):
        idx = torch.arange(cap - 3, cap, device="cuda", dtype=torch.int32).expand(2, 3).contiguous()
        assert torch.equal(csa.csa2_cache_read(c, idx, keys=keys), csa.csa2_cache_read(small, first=5, count=3, keys=keys))


# ---------------------------------------------------------------- reading back

def filled(csa, B, cap, d_idx, seed=0):
    g = gen(seed)
    return csa.Cache.of(*fp4((B, cap, 512), g), *fp4((B, cap, d_idx), g), ratio=1)


@pytest.mark.parametrize("dtype", [BF, HF, F])
@pytest.mark.parametrize("d_idx", [64, 128])
@pytest.mark.parametrize("keys", [False, True])
def test_read_types(csa, dtype, d_idx, keys):
    c = filled(csa, 3, 77, d_idx)
    want = decode(c.ikey_codes, c.ikey_scales) if keys else decode(c.lat_codes, c.lat_scales)
    got = csa.csa2_cache_read(c, keys=keys, out_dtype=dtype)
    assert got.dtype == dtype and torch.equal(got.double(), want)
    got = csa.csa2_cache_read(c, first=5, count=33, keys=keys, out_dtype=dtype)
    assert torch.equal(got.double(), want[:, 5:38])


@pytest.mark.parametrize("n", [1, 2, 3, 31, 32, 33, 1000, 40000])
@pytest.mark.parametrize("dtype", [BF, F])
def test_read_lists(csa, n, dtype):
    g = gen(n)
    c = filled(csa, 3, 500, 128)
    idx = torch.randint(-3, 503, (3, n), generator=g, device="cuda", dtype=torch.int32)
    idx[0, 0], idx[1, 0], idx[2, 0] = (1 << 31) - 1, -(1 << 31), 499
    ok = ((idx >= 0) & (idx < 500))[..., None]
    b = torch.arange(3, device="cuda")[:, None]
    for keys in (False, True):
        want = decode(c.ikey_codes, c.ikey_scales) if keys else decode(c.lat_codes, c.lat_scales)
        want = torch.where(ok, want[b, idx.long().clamp(0, 499)], 0.0)
        got = csa.csa2_cache_read(c, idx, keys=keys, out_dtype=dtype)
        assert torch.equal(got.double(), want)


def test_read_every_code_and_scale(csa):
    """all 16 codes under all 256 scale bytes: exact in every type, NaN for the two bytes that are NaN"""
    codes = (torch.arange(8, device="cuda") * 2 + 16 * (torch.arange(8, device="cuda") * 2 + 1)).to(torch.uint8)
    c = csa.Cache.of(codes.repeat(32).expand(1, 8, 256).contiguous(), torch.arange(256, device="cuda").to(torch.uint8).view(1, 8, 32))
    want = decode(c.lat_codes, c.lat_scales)
    for dtype in (BF, HF, F):
        got = csa.csa2_cache_read(c, out_dtype=dtype).double()
        assert torch.equal(torch.isnan(got), torch.isnan(want)) and int(torch.isnan(got).sum()) == 32
        assert torch.equal(got.nan_to_num(0), want.nan_to_num(0))


def test_read_shapes_outputs_and_streams(csa):
    c = filled(csa, 2, 100, 64)
    idx = torch.randint(-1, 100, (2, 3, 7), generator=gen(1), device="cuda", dtype=torch.int32)
    got = csa.csa2_cache_read(c, idx)
    assert got.shape == (2, 3, 7, 512)
    assert torch.equal(got.view(2, 21, 512), csa.csa2_cache_read(c, idx.view(2, 21)))
    assert csa.csa2_cache_read(c, idx[:, :0]).shape == (2, 0, 7, 512) and csa.csa2_cache_read(c, first=100).shape == (2, 0, 512)
    guarded = torch.full((44, 512), 7.0, dtype=BF, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    csa.csa2_cache_read(c, idx, out=guarded[1:-1].view(2, 3, 7, 512), stream=s)
    s.synchronize()
    assert torch.equal(guarded[1:-1].view_as(got), got) and bool((guarded[0] == 7).all()) and bool((guarded[-1] == 7).all())


def test_append_and_read_in_a_graph(csa):
    """a captured step that appends at the device's positions and reads the entries back, replayed as they move on"""
    g = gen(2)
    B, n = 5, 3
    c = csa.Cache(B, 64, 128, ratio=2)
    ref = csa.Cache(B, 64, 128, ratio=2)
    rows, carried = randn((B, n, 512), g, BF), randn((B, 512), g, BF)
    w = [torch.rand(512, device="cuda", generator=g) for _ in range(2)]
    wik = fp4((128, 512), g)
    pos = torch.tensor([0, 1, 2, 31, 50], device="cuda")
    out = torch.empty((B, 64, 512), dtype=F, device="cuda")

    def step(cache, carry, o):
        csa.csa2_cache_append(cache, rows, pos, prev=carry, prev_out=carry, w0=w[0], w1=w[1], wik_codes=wik[0], wik_scales=wik[1])
        return csa.csa2_cache_read(cache, out=o)

    kept = carried.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(csa.Cache(B, 64, 128, ratio=2), kept.clone(), out)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(c, carried, out)
    for i in range(4):
        graph.replay()
        want = step(ref, kept, torch.empty_like(out))
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(carried, kept)
        for a, b in zip(planes(c), planes(ref)):
            assert torch.equal(a, b)
        pos += n
        rows.copy_(randn((B, n, 512), g, BF))


@pytest.mark.parametrize("d_idx", [64, 128])
@pytest.mark.parametrize("ratio", [1, 2])
def test_append_many_with_keys_along_paths(csa, ratio, d_idx):
    """as many entries as go through the tensor cores, of paths that end at once, in the middle, or not at all"""
    g = gen(12)
    path = torch.randint(0, 90, (4, 1600), generator=g, device="cuda", dtype=torch.int32)
    path[0, 1599] = -1
    path[1, 0] = 90
    path[2, 800:803] = -1
    append_case(csa, 4, 90, 1600, [7, 30, 1, 0], 1700, ratio=ratio, d_idx=d_idx, path=path, seed=13, alias=ratio == 2)


@pytest.mark.parametrize("d_idx", [64, 128])
def test_append_keys_next_to_their_thresholds(csa, d_idx):
    """rows and projections of few values, whose sums lie on the quantiser's thresholds or cancel to nothing; scales from
    the smallest to the largest in one row, whose small terms decide"""
    g = gen(14)
    B, R = 2, 1024
    for kind in range(5):
        rows = torch.zeros((B, R, 512), device="cuda")
        if kind == 0:
            rows += torch.randint(-1, 2, (B, R, 512), generator=g, device="cuda")
        elif kind == 1:
            rows[..., 0], rows[..., 16], rows[..., 32] = 448 * 6, 448 * 6, 2.0 ** -9 * torch.randint(1, 4, (B, R), generator=g, device="cuda")
        elif kind == 2:
            rows += torch.exp2(torch.randint(-14, 12, (B, R, 32), generator=g, device="cuda").float()).repeat_interleave(16, 2)
            rows *= torch.randint(0, 2, (B, R, 512), generator=g, device="cuda") * 2 - 1
        wc, ws = fp4((d_idx, 512), g)
        if kind == 0:
            wc, ws = torch.randint(0, 256, wc.shape, generator=g, device="cuda", dtype=torch.uint8) & 0xAA, torch.full_like(ws, 0x38)
        elif kind == 1:
            wc, ws = torch.full_like(wc, 0x77), torch.full_like(ws, 0x7E)
            wc[:, 8:16] = 0xFF                                       # cancels the first group against the second
        elif kind == 2:
            ws = torch.randint(0, 0x7F, ws.shape, generator=g, device="cuda", dtype=torch.uint8)
        elif kind == 3:                                              # the small term first, then two large ones that cancel
            rows[..., 16], rows[..., 32] = 448 * 6, 448 * 6
            rows[..., :16] = 2.0 ** -6 * torch.randint(-6, 7, (B, R, 16), generator=g, device="cuda")
            wc[:, 8:16], wc[:, 16:24] = 0x77, 0xFF
            ws[:, :1], ws[:, 1:] = 0x10, 0x7E
        rows = rows.to(BF)
        got, want = caches(csa, B, R, d_idx, 1), caches(csa, B, R, d_idx, 1)
        csa.csa2_cache_append(got, rows, torch.zeros(B, device="cuda", dtype=torch.int64), wik_codes=wc, wik_scales=ws)
        csa.csa2_cache_write_projected(want, rows, 0, None, None, wc, ws)
        for a, w in zip(planes(got), planes(want)):
            assert torch.equal(a, w)
