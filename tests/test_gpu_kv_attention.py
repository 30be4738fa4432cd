"""qknorm_kv_attention on the GPU against attention in 64 bits over the same cache bytes."""
import math

import pytest
import torch

import qk_norm_amd as q
from lowbit_ref import attention, random_cache

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


def make(lens, new, hq, hkv, D, dtype, seed, extra_pages=2, vscale=1.0, tail=0):
    """Rows of Q (and `tail` rows of no sequence after them), a cache and its page table."""
    g = torch.Generator().manual_seed(seed)
    need = [(n + 63) // 64 for n in lens]
    pages = sum(need) + extra_pages
    cache = random_cache(pages, hkv, D, seed + 1, vscale)
    order = torch.randperm(pages, generator=g)
    width = max([1] + need)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n].int()
        at += n
    starts = [0]
    for m in new:
        starts.append(starts[-1] + m)
    rows = torch.randn(starts[-1] + tail, (hq + 2 * hkv) * D, generator=g).to(dtype)
    return rows, cache, table, starts


def run(rows, cache, table, lens, starts, hq, hkv, D, dtype, scale=None, window=0, decode=False, want_lse=True,
        fill=3.0):
    T, B = rows.shape[0], len(lens)
    out = torch.full((T, hq * D + 8), fill, dtype=dtype, device="cuda")
    lse = torch.full((T, hq), fill, device="cuda") if want_lse else None
    need = q.qknorm_kv_attention_workspace_bytes(T, B, table.shape[1], hq, hkv, D)
    space = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    q.qknorm_kv_attention(rows.cuda(), cache.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                          out[:, :hq * D], hq, hkv, D, scale=scale,
                          q_starts=None if decode else torch.tensor(starts, dtype=torch.int32, device="cuda"),
                          window=window, lse=lse, workspace=space[:need])
    torch.cuda.synchronize()
    assert bool((out[:, hq * D:] == fill).all()) and bool((space[need:] == 0xFF).all())
    return out[:, :hq * D].cpu().view(T, hq, D), None if lse is None else lse.cpu()


def check(got, lse, rows, cache, table, lens, starts, hq, hkv, D, dtype, scale=None, window=0, fill=3.0):
    o, l, tol, ltol, covered = attention(rows, cache, table, lens, starts, hq, hkv, D, scale or D ** -0.5, window, dtype)
    err = (got.double() - o).abs()[covered]
    bad = ~(err <= tol[covered])
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} outputs off, worst {float((err / (tol[covered] + 1e-300)).max()):.2f} "
                           f"times the bound, first at {torch.nonzero(bad)[0].tolist()}")
    assert bool((got[~covered] == fill).all())
    if lse is not None:
        none = torch.isinf(l)
        assert torch.equal(torch.isinf(lse.double())[covered], none[covered])
        ok = covered[:, None] & ~none
        assert bool(((lse.double() - l).abs()[ok] <= ltol[ok]).all())
        assert bool((lse[~covered] == fill).all())


CASES = [
    # lens, new, hq, hkv, D, dtype, window
    ([1], [1], 1, 1, 64, BF, 0),
    ([63], [1], 4, 2, 128, HF, 0),
    ([64], [1], 8, 1, 128, BF, 0),
    ([65], [1], 3, 3, 256, BF, 0),
    ([0, 1, 129, 0], [1, 1, 1, 1], 6, 2, 64, HF, 0),
    ([257, 1000, 5, 64], [1, 1, 1, 1], 8, 2, 128, BF, 0),
    ([700, 333], [1, 1], 10, 2, 256, HF, 0),
    ([300], [7], 5, 1, 64, BF, 0),
    ([300, 80, 9], [3, 0, 9], 8, 2, 128, BF, 0),
    ([40, 10], [17, 10], 14, 2, 64, HF, 0),
    ([3], [5], 4, 2, 128, BF, 0),                         # two rows before the cache's first token see nothing
    ([200], [33], 4, 4, 128, BF, 0),
    ([500], [100], 6, 3, 64, BF, 0),
    ([150], [70], 4, 1, 256, HF, 0),
    ([300, 640], [1, 1], 4, 2, 128, BF, 1),
    ([300, 640], [1, 1], 4, 2, 128, HF, 64),
    ([300, 70, 1], [5, 20, 1], 7, 1, 64, BF, 33),
    ([2000], [3], 2, 1, 128, BF, 500),
    # more than 64 rows a sequence on average: the kernel of prompt chunks
    ([700, 90, 0, 300], [90, 90, 40, 1], 8, 2, 128, BF, 0),
    ([1000], [200], 4, 2, 64, HF, 100),
    ([260, 500], [130, 77], 6, 2, 256, BF, 64),
    ([50], [60], 8, 2, 128, HF, 0),
    ([129, 64, 1], [129, 64, 1], 3, 1, 64, BF, 0),
    ([2100], [65], 5, 1, 128, BF, 0),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_against_definition(case):
    lens, new, hq, hkv, D, dtype, window = CASES[case]
    print(f"[kv attention] {CASES[case]}", flush=True)
    rows, cache, table, starts = make(lens, new, hq, hkv, D, dtype, 50 + case, tail=2)
    got, lse = run(rows, cache, table, lens, starts, hq, hkv, D, dtype, window=window)
    check(got, lse, rows, cache, table, lens, starts, hq, hkv, D, dtype, window=window)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_decode_of_many_ragged_sequences(D):
    hq, hkv = 6, 2
    lens = [(i * 37) % 400 for i in range(70)]
    print(f"[kv attention] 70 sequences D={D}", flush=True)
    rows, cache, table, starts = make(lens, [1] * 70, hq, hkv, D, BF, D)
    got, lse = run(rows, cache, table, lens, starts, hq, hkv, D, BF, decode=True)
    check(got, lse, rows, cache, table, lens, starts, hq, hkv, D, BF)
    again, _ = run(rows, cache, table, lens, starts, hq, hkv, D, BF, decode=True, want_lse=False)
    assert torch.equal(got, again)


def test_one_long_sequence_among_short_ones():
    hq, hkv, D = 4, 1, 64
    lens = [5, 9000, 1, 64, 0, 130]
    print("[kv attention] one long among short", flush=True)
    rows, cache, table, starts = make(lens, [1, 2, 1, 1, 1, 3], hq, hkv, D, BF, 8)
    got, lse = run(rows, cache, table, lens, starts, hq, hkv, D, BF)
    check(got, lse, rows, cache, table, lens, starts, hq, hkv, D, BF)


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("vscale", [1e-25, 1e-4, 1e3, 1e25])
def test_values_of_any_magnitude(vscale, dtype):
    # V's scales far below fp16's range, and far above one (an fp16 output holds up to 65504)
    if dtype == HF and vscale > 1e3:
        pytest.skip("outputs would be infinite")
    hq, hkv, D, lens = 4, 2, 128, [260, 77]
    print(f"[kv attention] V scales about {vscale}", flush=True)
    rows, cache, table, starts = make(lens, [1, 1], hq, hkv, D, dtype, 21, vscale=vscale)
    got, lse = run(rows, cache, table, lens, starts, hq, hkv, D, dtype)
    check(got, lse, rows, cache, table, lens, starts, hq, hkv, D, dtype)


@pytest.mark.parametrize("scale", [1.0, 0.0, -0.3])
def test_scores_that_grow_along_the_cache(scale):
    # with scale 1 the scores span tens of powers of two and the maximum moves often
    hq, hkv, D, lens = 4, 2, 128, [900]
    print(f"[kv attention] scale={scale}", flush=True)
    rows, cache, table, starts = make(lens, [1], hq, hkv, D, BF, 33)
    got, lse = run(rows, cache, table, lens, starts, hq, hkv, D, BF, scale=scale)
    o, l, tol, ltol, _ = attention(rows, cache, table, lens, starts, hq, hkv, D, scale, 0, BF)
    assert bool(((got.double() - o).abs() <= tol).all()) and bool(((lse.double() - l).abs() <= ltol).all())


def test_hidden_places_may_hold_anything():
    # past the length, after a row's own token, outside the window, and pages that are not there
    hq, hkv, D, dtype = 4, 2, 128, BF
    lens, new, window = [100, 300], [4, 1], 90
    rows, cache, table, starts = make(lens, new, hq, hkv, D, dtype, 61)
    clean, clse = run(rows, cache, table, lens, starts, hq, hkv, D, dtype, window=window)
    nan = torch.tensor([math.nan, math.inf, -math.inf, 1e38]).to(BF).view(torch.uint8)

    def spoil(b, toks):
        for t in toks:
            p = int(table[b, t // 64])
            for at in (64 * D, 64 * D + 128):
                i = 2 * (t % 4)
                cache[p, :, at + 2 * (t % 64):at + 2 * (t % 64) + 2] = nan[i:i + 2]

    spoil(0, list(range(100, 128)) + list(range(0, 7)))        # row 0 of sequence 0 is token 96: sees 7..96
    spoil(1, list(range(300, 320)) + list(range(0, 210)))
    print("[kv attention] hidden places", flush=True)
    got, lse = run(rows, cache, table, lens, starts, hq, hkv, D, dtype, window=window)
    assert torch.equal(got, clean) and torch.equal(lse, clse)
    # a visible NaN reaches the rows that see it and no other
    spoil(0, [98])                                             # 98 % 4 == 2: -inf scale
    p = int(table[0, 1])
    cache[p, :, 64 * D + 2 * 34:64 * D + 2 * 34 + 2] = nan[0:2]
    got, lse = run(rows, cache, table, lens, starts, hq, hkv, D, dtype, window=window)
    assert torch.equal(got[:2], clean[:2]) and bool(got[2:4].isnan().all()) and torch.equal(got[4], clean[4])


def test_hidden_places_of_a_prompt_chunk_may_hold_anything():
    hq, hkv, D, dtype, window = 4, 1, 128, BF, 90
    lens, new = [200], [100]                                   # row 0 is token 100: sees 11..100; all rows see 110..100
    rows, cache, table, starts = make(lens, new, hq, hkv, D, dtype, 62)
    clean, clse = run(rows, cache, table, lens, starts, hq, hkv, D, dtype, window=window)
    check(clean, clse, rows, cache, table, lens, starts, hq, hkv, D, dtype, window=window)
    bad = cache.clone()
    nan = torch.tensor([math.nan, math.inf, -math.inf, 1e38]).to(BF).view(torch.uint8)
    for t in list(range(200, 256)) + list(range(0, 11)) + [150]:
        p = int(table[0, t // 64])
        for at in (64 * D, 64 * D + 128):
            bad[p, :, at + 2 * (t % 64):at + 2 * (t % 64) + 2] = nan[2 * (t % 4):2 * (t % 4) + 2] if t != 150 else nan[:2]
    print("[kv attention] hidden places of a chunk", flush=True)
    got, lse = run(rows, bad, table, lens, starts, hq, hkv, D, dtype, window=window)
    # token 150 (row 50) is seen by rows 50 .. 99
    assert torch.equal(got[:50], clean[:50]) and torch.equal(lse[:50], clse[:50])
    assert bool(got[50:].isnan().all())


@pytest.mark.parametrize("vscale", [1e-25, 1e-4, 1e25])
def test_prompt_chunk_with_values_of_any_magnitude(vscale):
    hq, hkv, D, dtype, lens = 4, 2, 64, BF, [150]
    print(f"[kv attention] chunk, V scales about {vscale}", flush=True)
    rows, cache, table, starts = make(lens, [100], hq, hkv, D, dtype, 63, vscale=vscale)
    got, lse = run(rows, cache, table, lens, starts, hq, hkv, D, dtype)
    check(got, lse, rows, cache, table, lens, starts, hq, hkv, D, dtype)


def test_pages_that_are_not_there_hide_a_prompt_chunks_tokens():
    hq, hkv, D, dtype, lens = 4, 2, 64, HF, [400, 200]
    rows, cache, table, starts = make(lens, [150, 80], hq, hkv, D, dtype, 72)
    table[0, 1], table[0, 4], table[1, :] = -1, cache.shape[0], 2 ** 31 - 1
    print("[kv attention] chunk, pages that are not there", flush=True)
    got, lse = run(rows, cache, table, lens, starts, hq, hkv, D, dtype)
    check(got, lse, rows, cache, table, lens, starts, hq, hkv, D, dtype)


def test_pages_that_are_not_there_hide_their_tokens():
    hq, hkv, D, dtype, lens = 4, 1, 64, HF, [400, 130]
    rows, cache, table, starts = make(lens, [2, 1], hq, hkv, D, dtype, 71)
    table[0, 1], table[0, 4], table[1, :] = -1, cache.shape[0], 2 ** 31 - 1
    print("[kv attention] pages that are not there", flush=True)
    got, lse = run(rows, cache, table, lens, starts, hq, hkv, D, dtype)
    check(got, lse, rows, cache, table, lens, starts, hq, hkv, D, dtype)
    assert not got[2].any() and bool(torch.isinf(lse[2]).all())


def test_lengths_and_offsets_out_of_range_stay_inside():
    # lengths past the table and row offsets past the rows are taken at the bound
    hq, hkv, D, dtype = 2, 1, 64, BF
    rows, cache, table, _ = make([128, 128], [1, 1], hq, hkv, D, dtype, 81)
    print("[kv attention] out of range", flush=True)
    a = run(rows, cache, table, [1000, -5], [0, 1, 9], hq, hkv, D, dtype)
    b = run(rows, cache, table, [128, 0], [0, 1, 2], hq, hkv, D, dtype)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_no_pages_and_no_tokens():
    D = 64
    rows = torch.randn(2, 3 * D).to(BF)
    print("[kv attention] no pages", flush=True)
    got, lse = run(rows, torch.zeros(0, 1, 64 * D + 256, dtype=torch.uint8), torch.zeros(2, 3, dtype=torch.int32), [9, 0],
                   [0, 1, 2], 1, 1, D, BF)
    assert not got.any() and bool((lse == -math.inf).all())
    got, lse = run(rows, random_cache(1, 1, D, 1), torch.zeros(2, 0, dtype=torch.int32), [9, 0], [0, 1, 2], 1, 1, D, BF)
    assert not got.any() and bool((lse == -math.inf).all())


def test_past_four_gib():
    hq, hkv, D = 4, 8, 128
    hq = 8
    per = q.qknorm_kv_page_bytes(hkv, D)
    pages = (1 << 32) // per + 40
    print(f"[kv attention] {pages * per / 2 ** 30:.2f} GiB of pages", flush=True)
    few = random_cache(12, hkv, D, 3)
    cache = torch.empty(pages, hkv, 64 * D + 256, dtype=torch.uint8, device="cuda")
    far = [pages - 1 - 3 * i for i in range(11)] + [0]
    cache[far] = few.cuda()
    g = torch.Generator().manual_seed(4)
    rows = torch.randn(2, (hq + 2 * hkv) * D, generator=g).to(BF)
    lens, starts = [380, 361], [0, 1, 2]
    near = torch.tensor([[0, 1, 2, 3, 4, 5], [6, 7, 8, 9, 10, 11]], dtype=torch.int32)
    got, lse = run(rows, cache, torch.tensor(far, dtype=torch.int32).view(2, 6), lens, starts, hq, hkv, D, BF)
    check(got, lse, rows, few, near, lens, starts, hq, hkv, D, BF)


def test_replayed_graph_takes_lengths_and_offsets_of_the_day():
    hq, hkv, D, dtype = 8, 2, 128, BF
    lens, new = [900, 40, 300], [1, 1, 1]
    rows, cache, table, starts = make(lens, new, hq, hkv, D, dtype, 91)
    r, c, t = rows.cuda(), cache.cuda(), table.cuda()
    L = torch.tensor(lens, dtype=torch.int32, device="cuda")
    S = torch.tensor(starts, dtype=torch.int32, device="cuda")
    out = torch.zeros(3, hq, D, dtype=dtype, device="cuda")
    lse = torch.zeros(3, hq, device="cuda")
    space = torch.empty(q.qknorm_kv_attention_workspace_bytes(3, 3, t.shape[1], hq, hkv, D), dtype=torch.uint8, device="cuda")
    call = lambda: q.qknorm_kv_attention(r, c, t, L, out, hq, hkv, D, q_starts=S, lse=lse, workspace=space)  # noqa: E731
    print("[kv attention] graph", flush=True)
    call()
    torch.cuda.synchronize()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        call()
    torch.cuda.synchronize()
    for now, st in (([900, 40, 300], [0, 1, 2, 3]), ([1, 0, 257], [0, 0, 2, 3]), ([640, 33, 128], [0, 2, 2, 3])):
        L.copy_(torch.tensor(now, dtype=torch.int32))
        S.copy_(torch.tensor(st, dtype=torch.int32))
        out.fill_(3.0)
        lse.fill_(3.0)
        space.fill_(0x5A)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check(out.cpu(), lse.cpu(), rows, cache, table, now, st, hq, hkv, D, dtype)
        got, glse = out.clone(), lse.clone()
        call()
        torch.cuda.synchronize()
        assert torch.equal(out, got) and torch.equal(lse, glse)


def test_two_streams_with_workspaces_of_their_own():
    hq, hkv, D, dtype = 8, 2, 128, BF
    sets = [make([3000, 10], [1, 1], hq, hkv, D, dtype, 200 + i) for i in range(2)]
    want = [run(*s[:3], [3000, 10], s[3], hq, hkv, D, dtype)[0] for s in sets]
    dev = []
    for rows, cache, table, starts in sets:
        space = torch.empty(q.qknorm_kv_attention_workspace_bytes(2, 2, table.shape[1], hq, hkv, D), dtype=torch.uint8,
                            device="cuda")
        dev.append((rows.cuda(), cache.cuda(), table.cuda(), torch.tensor([3000, 10], dtype=torch.int32, device="cuda"),
                    torch.zeros(2, hq, D, dtype=dtype, device="cuda"), space, torch.cuda.Stream()))
    torch.cuda.synchronize()
    print("[kv attention] two streams", flush=True)
    for _ in range(5):
        for rows, cache, table, L, out, space, st in dev:
            q.qknorm_kv_attention(rows, cache, table, L, out, hq, hkv, D, workspace=space, stream=st)
    torch.cuda.synchronize()
    for d, w in zip(dev, want):
        assert torch.equal(d[4].cpu(), w)


def test_heads_that_share_keys_agree():
    # the same query in every head of a group gives the same output in each
    hq, hkv, D = 12, 3, 64
    rows, cache, table, starts = make([200], [4], hq, hkv, D, BF, 17)
    x = rows[:, :hq * D].view(4, hkv, 4, D)
    x[:] = x[:, :, :1]
    print("[kv attention] shared heads", flush=True)
    got, _ = run(rows, cache, table, [200], starts, hq, hkv, D, BF)
    got = got.view(4, hkv, 4, D)
    assert torch.equal(got, got[:, :, :1].expand_as(got))


@pytest.mark.parametrize("D,B,hkv", [(256, 520, 8), (64, 4096, 2), (128, 780, 8)])
def test_decode_of_more_units_than_waves(D, B, hkv):
    # lengths 0 .. 90 on two pages a sequence; 520 sequences of 8 heads: each unit is one wave's
    lens = [(i * 53) % 91 for i in range(B)]
    print(f"[kv attention] {B} sequences, {hkv} heads, D={D}", flush=True)
    rows, cache, table, starts = make(lens, [1] * B, hkv, hkv, D, BF, D + B)
    got, lse = run(rows, cache, table, lens, starts, hkv, hkv, D, BF, decode=True)
    k = B // 130                                               # (every k-th against the definition)
    check(got[::k], lse[::k], rows[::k], cache, table[::k], lens[::k], list(range(len(lens[::k]) + 1)), hkv, hkv, D, BF)
    by_offsets, lse2 = run(rows, cache, table, lens, starts, hkv, hkv, D, BF)
    assert torch.equal(got, by_offsets) and torch.equal(lse, lse2)


def test_prompt_of_more_units_than_waves():
    # 16 heads of 32-row tiles: 130 tiles over 17 pages
    hq, hkv, D, n = 64, 16, 256, 1040
    print("[kv attention] long prompt", flush=True)
    rows, cache, table, starts = make([n], [n], hq, hkv, D, HF, 17)
    got, lse = run(rows, cache, table, [n], starts, hq, hkv, D, HF)
    some = [0, 1, 63, 64, 500, 1039]                           # (each row alone, as the last token of its own prefix)
    for i in some:
        lens = [i + 1]
        o, l, tol, ltol, _ = attention(rows[i:i + 1], cache, table, lens, [0, 1], hq, hkv, D, D ** -0.5, 0, HF)
        assert bool(((got[i:i + 1].double() - o).abs() <= tol).all()) and bool(((lse[i:i + 1].double() - l).abs() <= ltol).all())
    assert bool(torch.isfinite(got).all()) and bool(torch.isfinite(lse).all())


@pytest.mark.parametrize("new", [[5, 3], [70, 40]], ids=["few", "many"])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_a_row_of_q_that_is_not_finite_stays_alone(value, new):
    hq, hkv, D, dtype, lens = 4, 1, 128, BF, [200, 100]
    rows, cache, table, starts = make(lens, new, hq, hkv, D, dtype, 91)
    rows[2, 5] = value                                         # row 2, query head 0
    print(f"[kv attention] {value} in Q", flush=True)
    got, lse = run(rows, cache, table, lens, starts, hq, hkv, D, dtype)
    assert bool(got[2, 0].isnan().all()) and bool(lse[2, 0].isnan())
    rows[2, 5] = 0
    o, l, tol, ltol, _ = attention(rows, cache, table, lens, starts, hq, hkv, D, D ** -0.5, 0, dtype)
    rest = torch.ones(rows.shape[0], hq, dtype=torch.bool)
    rest[2, 0] = False
    assert bool(((got.double() - o).abs() <= tol)[rest].all()) and bool(((lse.double() - l).abs() <= ltol)[rest].all())


def test_row_offsets_out_of_order_touch_nothing_else():
    # rows of sequences with offsets in order keep their results; run() checks what lies around out and workspace
    hq, hkv, D, dtype = 4, 2, 64, BF
    lens = [70, 40, 130, 64]
    rows, cache, table, _ = make(lens, [2, 2, 2, 2], hq, hkv, D, dtype, 95)
    print("[kv attention] offsets out of order", flush=True)
    for starts in ([0, 8, 0, 8, 0], [8, 6, 4, 2, 0], [-3, 100, -7, 50, 2], [2 ** 31 - 1, -2 ** 31, 4, 4, 4]):
        run(rows, cache, table, lens, starts, hq, hkv, D, dtype)


# Page tables much wider than the sequences need: those calls split units over waves that know nothing of one
# another, where the ones above mostly give each to a block.
WIDE = ([(test_against_definition, (i,)) for i in range(len(CASES))]
        + [(test_values_of_any_magnitude, a) for a in ((1e-25, BF), (1e25, BF), (1e3, HF))]
        + [(test_scores_that_grow_along_the_cache, (a,)) for a in (1.0, -0.3)]
        + [(test_prompt_chunk_with_values_of_any_magnitude, (a,)) for a in (1e-25, 1e25)]
        + [(test_a_row_of_q_that_is_not_finite_stays_alone, a) for a in ((math.nan, [5, 3]), (math.inf, [70, 40]))]
        + [(f, ()) for f in (test_hidden_places_may_hold_anything, test_hidden_places_of_a_prompt_chunk_may_hold_anything,
                             test_pages_that_are_not_there_hide_a_prompt_chunks_tokens,
                             test_pages_that_are_not_there_hide_their_tokens,
                             test_row_offsets_out_of_order_touch_nothing_else, test_heads_that_share_keys_agree)])


@pytest.mark.parametrize("which", range(len(WIDE)))
def test_wide_page_tables(which, monkeypatch):
    plain = make

    def wide(*args, **kw):
        rows, cache, table, starts = plain(*args, **kw)
        more = torch.full((table.shape[0], 600), 2 ** 31 - 1, dtype=torch.int32)
        return rows, cache, torch.cat([table, more], 1), starts

    f, args = WIDE[which]
    print(f"[kv attention] wide table: {f.__name__} {args}", flush=True)
    monkeypatch.setitem(globals(), "make", wide)
    f(*args)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,length,new,hkv", [(1, 130, 1, 1), (1, 900, 1, 2), (50, 300, 1, 8), (6, 600, 9, 3), (3, 520, 150, 2)])
def test_short_sequences(B, length, new, hkv, D):
    # four and eight waves a block, one and two row tiles; some sequences of other lengths, one of none
    lens = [max(0, length - 61 * i) for i in range(B)]
    rows_of = [min(new, 1 + i) if new > 1 and i else new for i in range(B)]
    print(f"[kv attention] short B={B} length={length} new={new} hkv={hkv} D={D}", flush=True)
    dtype = HF if D == 128 else BF
    hq = 4 * hkv
    rows, cache, table, starts = make(lens, rows_of, hq, hkv, D, dtype, B + length, tail=1)
    got, lse = run(rows, cache, table, lens, starts, hq, hkv, D, dtype)
    check(got, lse, rows, cache, table, lens, starts, hq, hkv, D, dtype)
    again, _ = run(rows, cache, table, lens, starts, hq, hkv, D, dtype, want_lse=False)
    assert torch.equal(got, again)


def check_rows(got, lse, some, rows, cache, table, hq, hkv, D, dtype):
    """Rows of one prompt that begins the cache, each as the last token of its own prefix."""
    for i in some:
        o, l, tol, ltol, _ = attention(rows[i:i + 1], cache, table, [i + 1], [0, 1], hq, hkv, D, D ** -0.5, 0, dtype)
        assert bool(((got[i:i + 1].double() - o).abs() <= tol).all()), i
        assert bool(((lse[i:i + 1].double() - l).abs() <= ltol).all()), i
    assert bool(torch.isfinite(got).all()) and bool(torch.isfinite(lse).all())


@pytest.mark.parametrize("D,dtype", [(64, HF), (128, BF)])
def test_prompt_of_a_wave_a_unit(D, dtype):
    heads, n = 64, 500
    print(f"[kv attention] prompt of 64 heads D={D}", flush=True)
    rows, cache, table, starts = make([n], [n], heads, heads, D, dtype, D)
    got, lse = run(rows, cache, table, [n], starts, heads, heads, D, dtype)
    check_rows(got, lse, [0, 31, 32, 100, 499], rows, cache, table, heads, heads, D, dtype)


def test_many_prompts():
    # more than 64 sequences, and more units of two row tiles than twice the waves
    hq, hkv, D, B, new = 32, 8, 256, 70, 40
    print("[kv attention] 70 prompts", flush=True)
    lens = [40 + (7 * i) % 50 for i in range(B)]
    rows, cache, table, starts = make(lens, [new] * B, hq, hkv, D, BF, 77)
    got, lse = run(rows, cache, table, lens, starts, hq, hkv, D, BF)
    for b in (0, 37, 69):
        lo, hi = starts[b], starts[b + 1]
        check(got[lo:hi], lse[lo:hi], rows[lo:hi], cache, table[b:b + 1], lens[b:b + 1], [0, new], hq, hkv, D, BF)
    assert bool(torch.isfinite(got).all()) and bool(torch.isfinite(lse).all())
