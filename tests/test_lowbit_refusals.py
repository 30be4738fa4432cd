"""What the 8-bit projection and the 4-bit cache's calls refuse, through the C ABI on the host (every argument is checked
before any GPU call, so these run without one), and through the binding."""
import ctypes

import pytest
import torch

import qk_norm_amd as q

OK, NULLP, SHAPE, ALIGN, DTYPE, UNSUP, EPS = 0, -1, -2, -3, -4, -5, -6
P = 1 << 20           # an aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    return q.load()


def call(lib, name, base, **changes):
    a = dict(base, **changes)
    return getattr(lib, name)(*a.values())


QUANT = dict(x=P, ldx=64, q=P, ldq=64, scale=P, T=2, n=64, dtype=q.QKNORM_BF16, stream=None)
PROJ = dict(x=P, ldx=128, xs=P, w=P, ldw=128, ws=P, qkv=P, ld=512, T=2, hidden=128, hq=2, hkv=1, head_dim=128, gq=P, gk=P,
            eps=1e-6, flags=0, dtype=q.QKNORM_BF16, work=None, bytes=0, stream=None)
APPEND = dict(qkv=P, T=2, ld=512, hq=2, hkv=1, head_dim=128, cache=P, pages=4, stride=8448, slots=P, dtype=q.QKNORM_F16,
              stream=None)
GATHER = dict(cache=P, pages=4, stride=8448, slots=P, T=2, hkv=1, head_dim=128, k=P, ldk=128, v=P, ldv=128,
              dtype=q.QKNORM_F32, stream=None)
ATTN = dict(qkv=P, T=3, ld=512, cache=P, pages=4, stride=8448, table=P, ldt=8, max_pages=8, lens=P, starts=P, B=2, out=P,
            ldo=256, lse=None, hq=2, hkv=1, head_dim=128, scale=0.1, window=0, dtype=q.QKNORM_BF16, work=P, bytes=1 << 40,
            stream=None)


@pytest.mark.parametrize("name,base,changes,code", [
    ("qknorm_quant_rows", QUANT, dict(dtype=9), DTYPE),
    ("qknorm_quant_rows", QUANT, dict(dtype=q.QKNORM_F32), UNSUP),
    ("qknorm_quant_rows", QUANT, dict(dtype=q.QKNORM_FP8_E4M3), UNSUP),
    ("qknorm_quant_rows", QUANT, dict(T=-1), SHAPE),
    ("qknorm_quant_rows", QUANT, dict(n=-16), SHAPE),
    ("qknorm_quant_rows", QUANT, dict(ldx=48), SHAPE),
    ("qknorm_quant_rows", QUANT, dict(ldq=48), SHAPE),
    ("qknorm_quant_rows", QUANT, dict(x=None), NULLP),
    ("qknorm_quant_rows", QUANT, dict(scale=None), NULLP),
    ("qknorm_quant_rows", QUANT, dict(x=P + 8), ALIGN),
    ("qknorm_quant_rows", QUANT, dict(q=P + 8), ALIGN),
    ("qknorm_quant_rows", QUANT, dict(scale=P + 2), ALIGN),
    ("qknorm_quant_rows", QUANT, dict(n=56), ALIGN),
    ("qknorm_quant_rows", QUANT, dict(ldx=68), ALIGN),
    ("qknorm_quant_rows", QUANT, dict(ldq=72), ALIGN),
    ("qknorm_quant_rows", QUANT, dict(T=1 << 24), UNSUP),
    ("qknorm_quant_rows", QUANT, dict(ldx=1 << 40), UNSUP),
    ("qknorm_quant_rows", QUANT, dict(T=0, x=None, q=None, scale=None), OK),
    ("qknorm_qkv_proj_quant", PROJ, dict(dtype=-1), DTYPE),
    ("qknorm_qkv_proj_quant", PROJ, dict(dtype=q.QKNORM_F32), UNSUP),
    ("qknorm_qkv_proj_quant", PROJ, dict(eps=float("nan")), EPS),
    ("qknorm_qkv_proj_quant", PROJ, dict(eps=-1.0), EPS),
    ("qknorm_qkv_proj_quant", PROJ, dict(flags=2), UNSUP),
    ("qknorm_qkv_proj_quant", PROJ, dict(hidden=0), SHAPE),
    ("qknorm_qkv_proj_quant", PROJ, dict(ldx=112), SHAPE),
    ("qknorm_qkv_proj_quant", PROJ, dict(ld=504), SHAPE),
    ("qknorm_qkv_proj_quant", PROJ, dict(hidden=96), UNSUP),
    ("qknorm_qkv_proj_quant", PROJ, dict(hidden=131072, ldx=131072, ldw=131072), UNSUP),
    ("qknorm_qkv_proj_quant", PROJ, dict(head_dim=32, ld=512), UNSUP),
    ("qknorm_qkv_proj_quant", PROJ, dict(x=None), NULLP),
    ("qknorm_qkv_proj_quant", PROJ, dict(xs=None), NULLP),
    ("qknorm_qkv_proj_quant", PROJ, dict(ws=None), NULLP),
    ("qknorm_qkv_proj_quant", PROJ, dict(gk=None), NULLP),
    ("qknorm_qkv_proj_quant", PROJ, dict(x=P + 8), ALIGN),
    ("qknorm_qkv_proj_quant", PROJ, dict(ldx=136), ALIGN),
    ("qknorm_qkv_proj_quant", PROJ, dict(ldw=136), ALIGN),
    ("qknorm_qkv_proj_quant", PROJ, dict(ld=516), ALIGN),
    ("qknorm_qkv_proj_quant", PROJ, dict(xs=P + 1), ALIGN),
    ("qknorm_qkv_proj_quant", PROJ, dict(ws=P + 2), ALIGN),
    ("qknorm_qkv_proj_quant", PROJ, dict(work=P + 4, bytes=1 << 30), ALIGN),
    ("qknorm_qkv_proj_quant", PROJ, dict(work=P, bytes=16), SHAPE),
    ("qknorm_qkv_proj_quant", PROJ, dict(work=P, bytes=-1), SHAPE),
    ("qknorm_qkv_proj_quant", PROJ, dict(T=0, x=None, w=None, qkv=None, xs=None, ws=None, gq=None, gk=None), OK),
    ("qknorm_kv_append", APPEND, dict(dtype=7), DTYPE),
    ("qknorm_kv_append", APPEND, dict(dtype=q.QKNORM_F32), UNSUP),
    ("qknorm_kv_append", APPEND, dict(head_dim=96, ld=512), UNSUP),
    ("qknorm_kv_append", APPEND, dict(ld=504), SHAPE),
    ("qknorm_kv_append", APPEND, dict(hkv=-1), SHAPE),
    ("qknorm_kv_append", APPEND, dict(pages=-1), SHAPE),
    ("qknorm_kv_append", APPEND, dict(stride=8432), SHAPE),
    ("qknorm_kv_append", APPEND, dict(stride=8456), ALIGN),
    ("qknorm_kv_append", APPEND, dict(cache=P + 8), ALIGN),
    ("qknorm_kv_append", APPEND, dict(slots=P + 4), ALIGN),
    ("qknorm_kv_append", APPEND, dict(ld=516), ALIGN),
    ("qknorm_kv_append", APPEND, dict(qkv=None), NULLP),
    ("qknorm_kv_append", APPEND, dict(slots=None), NULLP),
    ("qknorm_kv_append", APPEND, dict(cache=None), NULLP),
    ("qknorm_kv_append", APPEND, dict(T=1 << 29), UNSUP),
    ("qknorm_kv_append", APPEND, dict(pages=1 << 41), UNSUP),
    ("qknorm_kv_append", APPEND, dict(T=0, qkv=None, slots=None, cache=None), OK),
    ("qknorm_kv_append", APPEND, dict(hkv=0, qkv=None, slots=None), OK),
    ("qknorm_kv_gather", GATHER, dict(dtype=q.QKNORM_FP8_E4M3), UNSUP),
    ("qknorm_kv_gather", GATHER, dict(dtype=4), DTYPE),
    ("qknorm_kv_gather", GATHER, dict(ldk=124), SHAPE),
    ("qknorm_kv_gather", GATHER, dict(ldv=130), ALIGN),
    ("qknorm_kv_gather", GATHER, dict(k=P + 4), ALIGN),
    ("qknorm_kv_gather", GATHER, dict(v=None), NULLP),
    ("qknorm_kv_gather", GATHER, dict(head_dim=80), UNSUP),
    ("qknorm_kv_gather", GATHER, dict(T=0, k=None, v=None, slots=None), OK),
    ("qknorm_kv_attention", ATTN, dict(dtype=q.QKNORM_F32), UNSUP),
    ("qknorm_kv_attention", ATTN, dict(dtype=12), DTYPE),
    ("qknorm_kv_attention", ATTN, dict(hq=3, ld=512, ldo=512, hkv=2), SHAPE),
    ("qknorm_kv_attention", ATTN, dict(hkv=0), SHAPE),
    ("qknorm_kv_attention", ATTN, dict(head_dim=32), UNSUP),
    ("qknorm_kv_attention", ATTN, dict(ld=248), SHAPE),
    ("qknorm_kv_attention", ATTN, dict(ldo=248), SHAPE),
    ("qknorm_kv_attention", ATTN, dict(ldt=7), SHAPE),
    ("qknorm_kv_attention", ATTN, dict(window=-1), SHAPE),
    ("qknorm_kv_attention", ATTN, dict(scale=float("inf")), SHAPE),
    ("qknorm_kv_attention", ATTN, dict(starts=None), SHAPE),             # T 3, B 2
    ("qknorm_kv_attention", ATTN, dict(B=4097), UNSUP),
    ("qknorm_kv_attention", ATTN, dict(max_pages=(1 << 24) + 1, ldt=1 << 25), UNSUP),
    ("qknorm_kv_attention", ATTN, dict(T=1 << 30), UNSUP),
    ("qknorm_kv_attention", ATTN, dict(ld=516), ALIGN),
    ("qknorm_kv_attention", ATTN, dict(qkv=P + 2), ALIGN),
    ("qknorm_kv_attention", ATTN, dict(out=P + 8), ALIGN),
    ("qknorm_kv_attention", ATTN, dict(table=P + 2), ALIGN),
    ("qknorm_kv_attention", ATTN, dict(lens=P + 1), ALIGN),
    ("qknorm_kv_attention", ATTN, dict(lse=P + 2), ALIGN),
    ("qknorm_kv_attention", ATTN, dict(work=P + 8), ALIGN),
    ("qknorm_kv_attention", ATTN, dict(work=None), NULLP),
    ("qknorm_kv_attention", ATTN, dict(bytes=256), SHAPE),
    ("qknorm_kv_attention", ATTN, dict(lens=None), NULLP),
    ("qknorm_kv_attention", ATTN, dict(table=None), NULLP),
    ("qknorm_kv_attention", ATTN, dict(cache=None), NULLP),
    ("qknorm_kv_attention", ATTN, dict(stride=8000), SHAPE),
    ("qknorm_kv_attention", ATTN, dict(T=0, qkv=None, out=None), OK),
    ("qknorm_kv_attention", ATTN, dict(T=0, B=0, qkv=None, out=None, lens=None, table=None, work=None, bytes=0), OK),
])
def test_codes(lib, name, base, changes, code):
    assert call(lib, name, base, **changes) == code


def test_sizes(lib):
    assert q.qknorm_kv_page_bytes(8, 128) == 8 * 8448
    assert q.qknorm_kv_page_bytes(0, 64) == 0
    assert lib.qknorm_kv_page_bytes(1, 80) == UNSUP and lib.qknorm_kv_page_bytes(-1, 64) == SHAPE
    assert q.qknorm_qkv_proj_quant_workspace_bytes(65, 2, 1, 128) == 0
    assert q.qknorm_qkv_proj_quant_workspace_bytes(0, 2, 1, 128) == 0
    for T in (1, 8, 9, 16, 17, 32, 33, 64):
        assert q.qknorm_qkv_proj_quant_workspace_bytes(T, 2, 1, 128) >= T * 512 * 4
    assert lib.qknorm_qkv_proj_quant_workspace_bytes(-1, 2, 1, 128) == SHAPE
    assert lib.qknorm_kv_attention_workspace_bytes(1, 1, 1, 3, 2, 128) == SHAPE
    assert lib.qknorm_kv_attention_workspace_bytes(1, 5000, 1, 2, 2, 128) == UNSUP
    assert q.qknorm_kv_attention_workspace_bytes(0, 3, 9, 2, 2, 128) == 0
    assert lib.qknorm_kv_attention_workspace_bytes(2 ** 62, 1, 1, 2, 2, 128) == UNSUP
    assert lib.qknorm_kv_attention_workspace_bytes(1, 1, 2 ** 62, 2, 2, 128) == UNSUP
    assert ctypes.c_int64(q.qknorm_kv_attention_workspace_bytes(4096, 64, 4096, 64, 8, 256)).value < 1 << 30


def test_binding_refuses_cpu_tensors_and_wrong_types():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    i8, f = torch.zeros(2, 64, dtype=torch.int8), torch.zeros(2)
    cache = torch.zeros(1, 1, 64 * 64 + 256, dtype=torch.uint8)
    for fn in (lambda: q.qknorm_quant_rows(x, i8, f),
               lambda: q.qknorm_qkv_proj_quant(i8, f, i8, f, x, 1, 0, 64),
               lambda: q.qknorm_kv_append(x, 0, 1, 64, cache, torch.zeros(2, dtype=torch.int64)),
               lambda: q.qknorm_kv_gather(cache, torch.zeros(2, dtype=torch.int64), x, x, 1, 64),
               lambda: q.qknorm_kv_attention(x, cache, torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                                             x, 1, 1, 64)):
        with pytest.raises(ValueError, match="GPU"):
            fn()


@pytest.mark.gpu
def test_binding_refuses_wrong_gpu_arguments():
    d = dict(device="cuda")
    x = torch.zeros(2, 192, dtype=torch.bfloat16, **d)
    cache = torch.zeros(3, 1, 64 * 64 + 256, dtype=torch.uint8, **d)
    slots, lens = torch.zeros(2, dtype=torch.int64, **d), torch.zeros(2, dtype=torch.int32, **d)
    table, out = torch.zeros(2, 1, dtype=torch.int32, **d), torch.zeros(2, 64, dtype=torch.bfloat16, **d)
    work = torch.empty(q.qknorm_kv_attention_workspace_bytes(2, 2, 1, 1, 1, 64), dtype=torch.uint8, **d)
    i8, f = torch.zeros(2, 192, dtype=torch.int8, **d), torch.zeros(2, **d)
    bad = [
        lambda: q.qknorm_quant_rows(x, i8.to(torch.uint8), f),
        lambda: q.qknorm_quant_rows(x, i8[:, :64], f),
        lambda: q.qknorm_quant_rows(x, i8, f.double()),
        lambda: q.qknorm_quant_rows(x, i8, f[:1]),
        lambda: q.qknorm_quant_rows(x.float(), i8, f),
        lambda: q.qknorm_qkv_proj_quant(x, f, i8, f, x, 1, 1, 64),
        lambda: q.qknorm_qkv_proj_quant(i8, f, torch.zeros(100, 192, dtype=torch.int8, **d), torch.zeros(100, **d), x, 1, 1, 64),
        lambda: q.qknorm_kv_append(x, 1, 1, 64, cache, slots.int()),
        lambda: q.qknorm_kv_append(x, 1, 1, 64, cache, slots[:1]),
        lambda: q.qknorm_kv_append(x, 1, 1, 64, cache.view(torch.int8), slots),
        lambda: q.qknorm_kv_append(x, 1, 1, 64, cache[:, :, :4000], slots),
        lambda: q.qknorm_kv_append(x, 2, 1, 64, cache, slots),
        lambda: q.qknorm_kv_append(x, 1, 1, 64, cache, slots.cpu()),
        lambda: q.qknorm_kv_gather(cache, slots, out, out.float(), 1, 64),
        lambda: q.qknorm_kv_gather(cache, slots, out[:, :32], out[:, :32], 1, 64),
        lambda: q.qknorm_kv_attention(x, cache, table, lens, out, 1, 1, 64),                         # no workspace
        lambda: q.qknorm_kv_attention(x, cache, table, lens, out, 1, 1, 64, workspace=work[:64]),
        lambda: q.qknorm_kv_attention(x, cache, table.long(), lens, out, 1, 1, 64, workspace=work),
        lambda: q.qknorm_kv_attention(x, cache, table, lens[:1], out, 1, 1, 64, workspace=work),
        lambda: q.qknorm_kv_attention(x, cache, table, lens, out.half(), 1, 1, 64, workspace=work),
        lambda: q.qknorm_kv_attention(x, cache, table, lens, out[:, :32], 1, 1, 64, workspace=work),
        lambda: q.qknorm_kv_attention(x, cache, table, lens, out, 1, 1, 64, q_starts=lens, workspace=work),
        lambda: q.qknorm_kv_attention(x, cache, table, lens, out, 1, 1, 64, lse=f[:1], workspace=work),
        lambda: q.qknorm_kv_attention(x, cache, table, lens, out, 1, 1, 64, scale=float("nan"), workspace=work),
        lambda: q.qknorm_kv_attention(x, cache, table, lens, out, 1, 1, 64, window=-3, workspace=work),
    ]
    for i, fn in enumerate(bad):
        with pytest.raises(ValueError):
            fn()
            pytest.fail(f"call {i} was not refused")
    torch.cuda.synchronize()
    assert not out.any() and not cache.any()


@pytest.mark.gpu
def test_binding_refuses_rows_narrower_than_the_heads():
    # views whose pitch would do, but whose own columns would not; gamma of another length
    d = dict(device="cuda")
    wide = torch.zeros(2, 384, dtype=torch.bfloat16, **d)
    cache = torch.zeros(3, 1, 64 * 64 + 256, dtype=torch.uint8, **d)
    slots = torch.zeros(2, dtype=torch.int64, **d)
    x, w, f = torch.zeros(2, 64, dtype=torch.int8, **d), torch.zeros(192, 64, dtype=torch.int8, **d), torch.zeros(192, **d)
    g = torch.ones(128, dtype=torch.bfloat16, **d)
    bad = [
        lambda: q.qknorm_kv_append(wide[:, :128], 1, 1, 64, cache, slots),
        lambda: q.qknorm_qkv_proj_quant(x, f[:2], w, f, wide[:, :128], 1, 1, 64, plain=True),
        lambda: q.qknorm_qkv_proj_quant(x, f[:2], w, f, wide, 1, 1, 64, g[:32], g[:64]),
        lambda: q.qknorm_qkv_proj_quant(x, f[:2], w, f, wide, 1, 1, 64, g[:64], g),
    ]
    for i, fn in enumerate(bad):
        with pytest.raises(ValueError):
            fn()
            pytest.fail(f"call {i} was not refused")
    q.qknorm_qkv_proj_quant(x, f[:2], w, f, wide[:, :192], 1, 1, 64, g[:64], g[:64])
    torch.cuda.synchronize()
    assert not wide.any() and not cache.any()
