"""qknorm_qkv_proj_quant on the GPU against its definition in 64 bits, every tile shape and the workspace form."""
import pytest
import torch

import qk_norm_amd as q
from lowbit_ref import proj_quant, proj_tolerance

pytestmark = pytest.mark.gpu
EPS = 1e-6


def make(T, hidden, hq, hkv, D, dtype, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    N = (hq + 2 * hkv) * D
    x = torch.randint(-127, 128, (T, hidden + pad), generator=g, dtype=torch.int8)
    w = torch.randint(-127, 128, (N, hidden + pad), generator=g, dtype=torch.int8)
    xs = torch.rand(T, generator=g) * 0.05 + 1e-3
    ws = torch.rand(N, generator=g) * 1e-3 + 1e-5
    gq = (torch.rand(D, generator=g) + 0.5).to(dtype)
    gk = (torch.rand(D, generator=g) + 0.5).to(dtype)
    return x, xs, w, ws, gq, gk


def run(x, xs, w, ws, gq, gk, hidden, hq, hkv, D, dtype, plain, space, pad_out=0):
    T, N = x.shape[0], w.shape[0]
    out = torch.full((T, N + pad_out), 7.0, dtype=dtype, device="cuda")
    need = q.qknorm_qkv_proj_quant_workspace_bytes(T, hq, hkv, D) if space else 0
    work = torch.empty(need, dtype=torch.uint8, device="cuda") if space else None
    q.qknorm_qkv_proj_quant(x.cuda()[:, :hidden], xs.cuda(), w.cuda()[:, :hidden], ws.cuda(), out, hq, hkv, D, gq.cuda(),
                            gk.cuda(), EPS, plain=plain, workspace=work)
    torch.cuda.synchronize()
    assert bool((out[:, N:] == 7).all())
    return out[:, :N].cpu()


def check(got, x, xs, w, ws, gq, gk, hidden, hq, hkv, D, dtype, plain):
    want = proj_quant(x[:, :hidden], xs, w[:, :hidden], ws, hq, hkv, D, gq, gk, EPS, plain)
    err = (got.double() - want).abs()
    tol = proj_tolerance(want, dtype, D)
    bad = ~(err <= tol)
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} outputs off, worst {float((err / tol).max()):.2f} times the bound, "
                           f"first at {torch.nonzero(bad)[0].tolist()}")


# token counts at and about every change of tile; hidden with half a K step left over and without
@pytest.mark.parametrize("T,hidden,hq,hkv,D,dtype,plain", [
    (1, 64, 1, 1, 64, torch.bfloat16, False),
    (2, 192, 2, 1, 128, torch.float16, False),
    (17, 128, 3, 1, 64, torch.bfloat16, True),
    (64, 320, 2, 2, 128, torch.bfloat16, False),
    (65, 1024, 4, 2, 64, torch.float16, False),
    (200, 448, 1, 1, 256, torch.bfloat16, False),
    (256, 256, 5, 1, 128, torch.bfloat16, False),
    (257, 576, 3, 1, 128, torch.float16, False),
    (333, 192, 2, 1, 256, torch.bfloat16, False),
    (512, 128, 2, 0, 64, torch.bfloat16, False),
    (513, 640, 30, 8, 128, torch.bfloat16, False),
    (700, 192, 34, 7, 64, torch.float16, True),
    (1025, 320, 3, 1, 128, torch.bfloat16, False),
    (1100, 448, 4, 2, 256, torch.float16, False),
])
def test_tiles(T, hidden, hq, hkv, D, dtype, plain):
    print(f"[proj_quant] T={T} hidden={hidden} hq={hq} hkv={hkv} D={D} {dtype} plain={plain}", flush=True)
    a = make(T, hidden, hq, hkv, D, dtype, T * 31 + hidden)
    check(run(*a, hidden, hq, hkv, D, dtype, plain, False), *a, hidden, hq, hkv, D, dtype, plain)


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 17, 31, 32, 33, 48, 64])
@pytest.mark.parametrize("hidden,hq,hkv,D,dtype", [(64, 1, 1, 64, torch.bfloat16), (832, 6, 2, 128, torch.float16),
                                                   (4096, 3, 1, 256, torch.bfloat16)])
def test_workspace_form(T, hidden, hq, hkv, D, dtype):
    print(f"[proj_quant] workspace T={T} hidden={hidden} D={D}", flush=True)
    a = make(T, hidden, hq, hkv, D, dtype, T * 7 + hidden)
    for plain in (False, True):
        got = run(*a, hidden, hq, hkv, D, dtype, plain, True)
        check(got, *a, hidden, hq, hkv, D, dtype, plain)
        if plain:       # the integer sums are exact: the tiles give the same bits
            assert torch.equal(got, run(*a, hidden, hq, hkv, D, dtype, plain, False))


@pytest.mark.parametrize("T", [5, 90, 300])
def test_pitches(T):
    hidden, hq, hkv, D, dtype = 448, 2, 1, 128, torch.bfloat16
    print(f"[proj_quant] pitches T={T}", flush=True)
    a = make(T, hidden, hq, hkv, D, dtype, T, pad=80)      # what follows a row is not zero
    check(run(*a, hidden, hq, hkv, D, dtype, False, T <= 64, pad_out=24), *a, hidden, hq, hkv, D, dtype, False)


def test_largest_sums_and_scales_of_zero_and_nan():
    hidden, hq, hkv, D, dtype = 131008, 1, 1, 64, torch.float16
    x = torch.full((3, hidden), -128, dtype=torch.int8)
    w = torch.full((3 * D, hidden), -128, dtype=torch.int8)
    w[1::2] = 127
    xs = torch.tensor([2.0 ** -30, 0.0, float("nan")])
    ws = torch.full((3 * D,), 1.0)
    one = torch.ones(D, dtype=dtype)
    for space in (False, True):
        print(f"[proj_quant] largest sums, workspace={space}", flush=True)
        got = run(x, xs, w, ws, one, one, hidden, hq, hkv, D, dtype, True, space)
        want = proj_quant(x[:2], xs[:2], w, ws, hq, hkv, D, one, one, EPS, True)
        assert bool(((got[:2].double() - want).abs() <= proj_tolerance(want, dtype, D)).all())
        assert bool(got[2].isnan().all()) and not got[1].any()


def test_replayed_graph_with_other_calls_between():
    T, hidden, hq, hkv, D, dtype = 12, 256, 4, 1, 128, torch.bfloat16
    x, xs, w, ws, gq, gk = (t.cuda() for t in make(T, hidden, hq, hkv, D, dtype, 11))
    space = torch.empty(q.qknorm_qkv_proj_quant_workspace_bytes(T, hq, hkv, D), dtype=torch.uint8, device="cuda")
    out = torch.empty(T, w.shape[0], dtype=dtype, device="cuda")
    call = lambda o: q.qknorm_qkv_proj_quant(x, xs, w, ws, o, hq, hkv, D, gq, gk, EPS, workspace=space)  # noqa: E731
    print("[proj_quant] graph", flush=True)
    call(out)
    torch.cuda.synchronize()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        call(out)
    torch.cuda.synchronize()
    for _ in range(3):
        x.copy_(torch.randint(-127, 128, x.shape, dtype=torch.int8, device="cuda"))
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        again = torch.empty_like(out)
        call(again)
        torch.cuda.synchronize()
        assert torch.equal(out, again)
