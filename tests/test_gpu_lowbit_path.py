"""The operators together, as a decoding attention block runs them: rows to 8 bits, the 8-bit projection with QK-Norm,
K and V into the 4-bit cache, attention over it -- prefill, then tokens one at a time, then the same in a replayed graph."""
import pytest
import torch

import qk_norm_amd as q
from lowbit_ref import attention, proj_quant, proj_tolerance, quant_rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,D", [(torch.bfloat16, 128), (torch.float16, 64)], ids=["bf16", "f16"])
def test_prefill_then_decode(dtype, D):
    hidden, hq, hkv, B, steps = 512, 4, 2, 3, 3
    N = (hq + 2 * hkv) * D
    g = torch.Generator(device="cuda").manual_seed(7)
    w = (torch.randn(N, hidden, generator=g, device="cuda") * hidden ** -0.5).to(dtype)
    wq, ws = torch.empty(N, hidden, dtype=torch.int8, device="cuda"), torch.empty(N, device="cuda")
    q.qknorm_quant_rows(w, wq, ws)
    gq = (torch.rand(D, generator=g, device="cuda") + 0.5).to(dtype)
    gk = (torch.rand(D, generator=g, device="cuda") + 0.5).to(dtype)
    cache = torch.zeros(3 * B, hkv, 64 * D + 256, dtype=torch.uint8, device="cuda")
    table = torch.randperm(3 * B, generator=torch.Generator().manual_seed(1)).int().view(B, 3)
    tab = table.cuda()

    def block(h, lens, starts, slots, one):
        """One attention block over rows h, with every step checked against its definition on its own inputs."""
        T = h.shape[0]
        xq, xs = torch.empty(T, hidden, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
        q.qknorm_quant_rows(h, xq, xs)
        qkv = torch.empty(T, N, dtype=dtype, device="cuda")
        need = q.qknorm_qkv_proj_quant_workspace_bytes(T, hq, hkv, D)
        q.qknorm_qkv_proj_quant(xq, xs, wq, ws, qkv, hq, hkv, D, gq, gk, workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
        q.qknorm_kv_append(qkv, hq, hkv, D, cache, torch.tensor(slots, dtype=torch.int64, device="cuda"))
        out = torch.empty(T, hq, D, dtype=dtype, device="cuda")
        space = torch.empty(q.qknorm_kv_attention_workspace_bytes(T, B, 3, hq, hkv, D), dtype=torch.uint8, device="cuda")
        q.qknorm_kv_attention(qkv, cache, tab, torch.tensor(lens, dtype=torch.int32, device="cuda"), out, hq, hkv, D,
                              q_starts=None if one else torch.tensor(starts, dtype=torch.int32, device="cuda"), workspace=space)
        torch.cuda.synchronize()
        rq, rs = quant_rows(h)
        assert torch.equal(xq.cpu(), rq) and torch.equal(xs.cpu(), rs)
        y = proj_quant(rq, rs, wq, ws, hq, hkv, D, gq, gk, 1e-6, False)
        assert bool(((qkv.cpu().double() - y).abs() <= proj_tolerance(y, dtype, D)).all())
        o, _, tol, _, _ = attention(qkv, cache.cpu(), table, lens, starts, hq, hkv, D, D ** -0.5, 0, dtype)
        assert bool(((out.cpu().double() - o).abs() <= tol).all())
        return out

    place = lambda b, t: int(table[b, t // 64]) * 64 + t % 64  # noqa: E731
    lens = [70, 1, 33]
    starts = [0, 70, 71, 104]
    slots = [place(b, t) for b in range(B) for t in range(lens[b])]
    print("[lowbit path] prefill", flush=True)
    block(torch.randn(104, hidden, generator=g, device="cuda").to(dtype), lens, starts, slots, False)
    for step in range(steps):
        print(f"[lowbit path] decode {step}", flush=True)
        slots = [place(b, lens[b]) for b in range(B)]
        lens = [n + 1 for n in lens]
        block(torch.randn(B, hidden, generator=g, device="cuda").to(dtype), lens, [0, 1, 2, 3], slots, True)


def test_decode_step_in_a_replayed_graph():
    dtype, D, hidden, hq, hkv, B = torch.bfloat16, 128, 256, 4, 2, 2
    N = (hq + 2 * hkv) * D
    g = torch.Generator(device="cuda").manual_seed(8)
    w = torch.randn(N, hidden, generator=g, device="cuda").to(dtype)
    wq, ws = torch.empty(N, hidden, dtype=torch.int8, device="cuda"), torch.empty(N, device="cuda")
    q.qknorm_quant_rows(w, wq, ws)
    one = torch.ones(D, dtype=dtype, device="cuda")
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
    h = torch.zeros(B, hidden, dtype=dtype, device="cuda")
    slots = torch.zeros(B, dtype=torch.int64, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    xq, xs = torch.empty(B, hidden, dtype=torch.int8, device="cuda"), torch.empty(B, device="cuda")
    qkv = torch.empty(B, N, dtype=dtype, device="cuda")
    out = torch.empty(B, hq, D, dtype=dtype, device="cuda")
    w1 = torch.empty(q.qknorm_qkv_proj_quant_workspace_bytes(B, hq, hkv, D), dtype=torch.uint8, device="cuda")
    w2 = torch.empty(q.qknorm_kv_attention_workspace_bytes(B, B, 2, hq, hkv, D), dtype=torch.uint8, device="cuda")

    def step(cache):
        q.qknorm_quant_rows(h, xq, xs)
        q.qknorm_qkv_proj_quant(xq, xs, wq, ws, qkv, hq, hkv, D, one, one, workspace=w1)
        q.qknorm_kv_append(qkv, hq, hkv, D, cache, slots)
        q.qknorm_kv_attention(qkv, cache, table, lens, out, hq, hkv, D, workspace=w2)

    mine = torch.zeros(4, hkv, 64 * D + 256, dtype=torch.uint8, device="cuda")
    other = mine.clone()
    print("[lowbit path] graph", flush=True)
    step(mine.clone())
    torch.cuda.synchronize()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        step(mine)
    torch.cuda.synchronize()
    for t in range(4):
        h.copy_(torch.randn(B, hidden, generator=g, device="cuda").to(dtype))
        slots.copy_(torch.tensor([62 + t, 128 + t]))           # the first sequence crosses a page's end
        slots[0] = 62 + t
        lens.copy_(torch.tensor([63 + t, 1 + t], dtype=torch.int32))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        step(other)
        torch.cuda.synchronize()
        assert torch.equal(out, got) and torch.equal(mine, other)
