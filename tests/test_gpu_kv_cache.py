"""The 4-bit cache's writer and reader on the GPU against the format in 64 bits: the same values, byte by byte
where they are stored, and nothing else touched."""
import math

import pytest
import torch

import qk_norm_amd as q
from lowbit_ref import code_values, random_cache, read_page, vector_codes

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16]


def rows(T, hq, hkv, D, dtype, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, (hq + 2 * hkv) * D + pad, generator=g) * torch.exp2(torch.randn(T, 1, generator=g) * 3)
    return x.to(dtype)


def values(x, hq, hkv, D):
    """K and V values [T, hkv, D] in 64 bits that the cache is to hold for rows x."""
    out = []
    for lo in (hq, hq + hkv):
        c, s = vector_codes(x[:, lo * D:(lo + hkv) * D].reshape(-1, hkv, D))
        out.append(code_values(c) * s.double()[..., None])
    return out


def append(x, hq, hkv, D, cache, slots):
    q.qknorm_kv_append(x.cuda(), hq, hkv, D, cache, torch.tensor(slots, dtype=torch.int64, device="cuda"))
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", TYPES, ids=["bf16", "f16"])
@pytest.mark.parametrize("T,hq,hkv,D,pad", [(1, 2, 1, 64, 0), (16, 3, 2, 128, 8), (17, 0, 3, 256, 0), (150, 1, 2, 128, 0),
                                            (1100, 0, 1, 64, 16), (1025, 1, 1, 256, 0), (1090, 1, 2, 128, 0)])
def test_append_stores_the_format(T, hq, hkv, D, pad, dtype):
    print(f"[kv] append T={T} hq={hq} hkv={hkv} D={D} pad={pad} {dtype}", flush=True)
    x = rows(T, hq, hkv, D, dtype, T + D, pad)
    pages = (T + 63) // 64 + 3
    start = random_cache(pages, hkv, D, 1)
    cache = start.cuda()
    perm = torch.randperm(pages * 64, generator=torch.Generator().manual_seed(T))[:T].tolist()
    run = [(pages * 64 - T) // 2 + i for i in range(T)]
    for slots in (perm, run):
        c = cache.clone()
        append(x, hq, hkv, D, c, slots)
        k, v = values(x, hq, hkv, D)
        got = [read_page(p, D) for p in c.cpu()]
        was = [read_page(p, D) for p in start]
        at = {s: i for i, s in enumerate(slots)}
        for page in range(pages):
            for t in range(64):
                i = at.get(page * 64 + t)
                wk, wv = (k[i], v[i]) if i is not None else (was[page][0][:, t], was[page][1][:, t])
                assert torch.equal(got[page][0][:, t], wk) and torch.equal(got[page][1][:, t], wv), (page, t, i)


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,hkv,D,pad", [(1, 1, 64, 0), (40, 2, 128, 8), (1030, 1, 256, 0), (1100, 3, 64, 16)])
def test_gather_reads_the_format(T, hkv, D, pad, out):
    print(f"[kv] gather T={T} hkv={hkv} D={D} {out}", flush=True)
    pages = 9
    host = random_cache(pages, hkv, D, T)
    page = [read_page(p, D) for p in host]
    g = torch.Generator().manual_seed(T)
    slots = torch.randint(-40, pages * 64 + 40, (T,), generator=g)          # repeated, negative and past the end
    k = torch.full((T, hkv * D + pad), 5.0, dtype=out, device="cuda")
    v = torch.full((T, hkv * D + pad), 6.0, dtype=out, device="cuda")
    q.qknorm_kv_gather(host.cuda(), slots.cuda(), k[:, :hkv * D], v[:, :hkv * D], hkv, D)
    torch.cuda.synchronize()
    assert bool((k[:, hkv * D:] == 5).all()) and bool((v[:, hkv * D:] == 6).all())
    k, v = k[:, :hkv * D].cpu().view(T, hkv, D), v[:, :hkv * D].cpu().view(T, hkv, D)
    for i, s in enumerate(slots.tolist()):
        if 0 <= s < pages * 64:
            assert torch.equal(k[i], page[s // 64][0][:, s % 64].to(out)), i
            assert torch.equal(v[i], page[s // 64][1][:, s % 64].to(out)), i
        else:
            assert bool((k[i] == 5).all()) and bool((v[i] == 6).all())


@pytest.mark.parametrize("dtype", TYPES, ids=["bf16", "f16"])
def test_halfway_points_extremes_and_non_finite_vectors(dtype):
    hkv, D = 1, 64
    big = float(torch.finfo(dtype).max)
    x = torch.zeros(12, 2 * D)
    half = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    near = torch.cat([half, half * (1 + 2.0 ** -7), half * (1 - 2.0 ** -7)])
    for i, e in enumerate((0.0, -9.0, 5.0)):                 # amax 6 * 2^e: scale 2^e exactly
        x[i, 0] = 6.0
        x[i, 1:22], x[i, 22:43] = near, -near
        x[i] *= 2.0 ** e
    x[3] = big
    x[4, 3], x[5, 4], x[6, 70] = math.inf, math.nan, -math.inf
    x[7] = 2.0 ** -24
    x[8] = 2.0 ** -110 if dtype == torch.bfloat16 else 2.0 ** -15
    x[9, :D] = torch.linspace(-7, 7, D)
    x[10, 0], x[10, 1] = 1e-30, 1.0
    x = x.to(dtype)
    print("[kv] halfway and extremes", flush=True)
    cache = random_cache(1, hkv, D, 2).cuda()
    append(x, 0, hkv, D, cache, list(range(20, 32)))
    k, v = values(x, 0, hkv, D)
    gk, gv = read_page(cache[0], D)
    for got, want in ((gk[:, 20:32].transpose(0, 1), k), (gv[:, 20:32].transpose(0, 1), v)):
        assert torch.equal(got.isnan(), want.isnan())
        assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))
    assert gk[0, 24].isnan().all() and gk[0, 25].isnan().all() and gv[0, 26].isnan().all() and not gk[0, 26].any()


def test_rows_without_a_place_are_skipped_and_pages_may_lie_apart():
    hq, hkv, D, T = 2, 2, 128, 30
    x = rows(T, hq, hkv, D, torch.bfloat16, 4)
    bytes_ = hkv * (64 * D + 256)
    pool = torch.full((3, 2, bytes_), 0xA5, dtype=torch.uint8, device="cuda")     # two layers' pages in turn
    cache = pool[:, 1].view(3, hkv, 64 * D + 256)
    slots = [5, -1, 3 * 64, 2 ** 40, -2 ** 40, 191] + [70 + i for i in range(T - 6)]
    print("[kv] slots without a place", flush=True)
    append(x, hq, hkv, D, cache, slots)
    assert bool((pool[:, 0] == 0xA5).all())
    k, v = values(x, hq, hkv, D)
    for i, s in enumerate(slots):
        if 0 <= s < 192:
            gk, gv = read_page(cache[s // 64], D)
            assert torch.equal(gk[:, s % 64], k[i]) and torch.equal(gv[:, s % 64], v[i])
    spare = cache[0].clone()
    spare[:, 5 * D // 2:6 * D // 2] = 0xA5                   # all of page 0 but token 5 is as it was
    for at in range(32 * D + 5, 64 * D, 64):
        spare[:, at] = 0xA5
    spare[:, 64 * D + 10:64 * D + 12] = 0xA5
    spare[:, 64 * D + 138:64 * D + 140] = 0xA5
    assert bool((spare == 0xA5).all())


def test_past_four_gib():
    hkv, D = 8, 128
    per = q.qknorm_kv_page_bytes(hkv, D)
    pages = (1 << 32) // per + 5
    print(f"[kv] {pages * per / 2 ** 30:.2f} GiB of pages", flush=True)
    cache = torch.empty(pages, hkv, 64 * D + 256, dtype=torch.uint8, device="cuda")
    x = rows(7, 1, hkv, D, torch.bfloat16, 9)
    slots = [(pages - 1 - i) * 64 + 63 - i for i in range(7)]
    append(x, 1, hkv, D, cache, slots)
    k = torch.zeros(7, hkv, D, device="cuda")
    v = torch.zeros(7, hkv, D, device="cuda")
    q.qknorm_kv_gather(cache, torch.tensor(slots, device="cuda"), k, v, hkv, D)
    torch.cuda.synchronize()
    wk, wv = values(x, 1, hkv, D)
    assert torch.equal(k.cpu().double(), wk) and torch.equal(v.cpu().double(), wv)


@pytest.mark.parametrize("T,hkv,D", [(4100, 2, 64), (4097, 1, 128), (4099, 1, 256)])
def test_many_rows_at_once(T, hkv, D):
    # rows of one call against the same rows 500 at a time, for places in order and apart
    dtype = torch.bfloat16
    print(f"[kv] {T} rows hkv={hkv} D={D}", flush=True)
    x = rows(T, 1, hkv, D, dtype, T).cuda()
    pages = (T + 63) // 64 + 2
    order = torch.randperm(pages * 64, generator=torch.Generator().manual_seed(D))[:T]
    for slots in (torch.arange(T) + 37, order):
        slots = slots.cuda()
        slots[::97] = -1
        one = random_cache(pages, hkv, D, 2).cuda()
        parts = one.clone()
        q.qknorm_kv_append(x, 1, hkv, D, one, slots)
        for i in range(0, T, 500):
            q.qknorm_kv_append(x[i:i + 500], 1, hkv, D, parts, slots[i:i + 500])
        assert torch.equal(one, parts)
        got = [torch.full((T, hkv * D), 7.0, dtype=dtype, device="cuda") for _ in range(4)]
        q.qknorm_kv_gather(one, slots, got[0], got[1], hkv, D)
        for i in range(0, T, 500):
            q.qknorm_kv_gather(one, slots[i:i + 500], got[2][i:i + 500], got[3][i:i + 500], hkv, D)
        torch.cuda.synchronize()
        for a, b in ((got[0], got[2]), (got[1], got[3])):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
        assert bool((got[0][::97] == 7).all())


def test_empty():
    c = torch.zeros(2, 1, 64 * 64 + 256, dtype=torch.uint8, device="cuda")
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    q.qknorm_kv_append(torch.empty(0, 128, dtype=torch.bfloat16, device="cuda"), 0, 1, 64, c, none)
    q.qknorm_kv_gather(c, none, torch.empty(0, 1, 64, device="cuda"), torch.empty(0, 1, 64, device="cuda"), 1, 64)
    torch.cuda.synchronize()
    assert not c.any()
