"""Refusals of the operators around the decode step, on the CPU: the C entry points' argument checks and the binding's."""

import ctypes

import pytest
import torch

import block_sparse_attention_attngate_b200 as S
from block_sparse_attention_attngate_b200 import seer

lib = seer._lib
P = ctypes.c_void_p(4096)       # aligned dummy addresses, never dereferenced on the host
ODD = ctypes.c_void_p(4100)


def said(word):
    return word in lib.seer_last_error().decode()


def reaches_cuda(call):
    """A well-formed call gets past the checks (only where no GPU would follow the dummy addresses)."""
    if not torch.cuda.is_available():
        assert call() == 4


def test_struct_layouts_match_c(tmp_path):
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    fields = {"seer_rows_t": S.RowsDesc, "seer_pool_t": S.PoolDesc, "seer_qk_t": S.QkShape, "seer_dense_t": S.DenseShape}
    lines = []
    for c, py in fields.items():
        lines.append(f'printf("%zu\\n", sizeof({c}));')
        lines += [f'printf("%zu\\n", offsetof({c}, {n}));' for n, _ in py._fields_]
    src = tmp_path / "l.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "seer.h"\nint main(void) {' + "\n".join(lines)
                   + 'printf("%d %d %d\\n", SEER_BF16, SEER_FP16, SEER_FP32); return 0; }\n')
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(root, "include"), str(src), "-o", str(tmp_path / "l")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "l")], capture_output=True, text=True, check=True).stdout.split()]
    want = []
    for py in fields.values():
        want.append(ctypes.sizeof(py))
        want += [getattr(py, n).offset for n, _ in py._fields_]
    assert got == want + [seer.DTYPES[torch.bfloat16], seer.DTYPES[torch.float16], seer.DTYPES[torch.float32]]


# ---------------------------------------------------------------- pages
def plan(batch=4, page=16, pages=64, width=8, room=32, **ptr):
    a = dict(lens=P, new=P, table=P, free=P, count=P, lo=P, co=P, cu=P, slots=P, pos=P)
    a.update(ptr)
    return lib.seer_page_plan(batch, page, pages, width, room, *a.values(), None, None)


def release(batch=4, page=16, pages=64, width=8, **ptr):
    a = dict(lens=P, done=P, table=P, free=P, count=P, lo=P, co=P)
    a.update(ptr)
    return lib.seer_page_release(batch, page, pages, width, *a.values(), None, None)


@pytest.mark.parametrize("call", [plan, release])
def test_page_call_refusals(call):
    for kw in (dict(batch=0), dict(page=0), dict(pages=0), dict(width=0)):
        assert call(**kw) == 1 and said(">= 1")
    assert call(batch=4097) == 2
    assert call(pages=1 << 20, page=1 << 11) == 2 and said("2^31")
    for name in ("lens", "table", "free", "count", "lo", "co"):
        assert call(**{name: None}) == 1 and said("NULL")
        assert call(**{name: ctypes.c_void_p(4098)}) == 1 and said("aligned")
    assert plan(room=0) == 1


def i32(*s):
    return torch.zeros(*s, dtype=torch.int32)


def refused(fn, good, name, bad, exc=ValueError):
    with pytest.raises(exc):
        fn(**{**good, name: bad})


def cuda_only(fn, good):
    with pytest.raises(TypeError, match="CUDA tensor"):
        fn(**good)


def test_page_binding_refusals():
    good = dict(page_size=16, seqlens=i32(4), new_tokens=i32(4), block_table=i32(4, 8), free_list=i32(64),
                free_count=i32(1), cu_tokens=i32(5), slot_map=i32(32), positions=i32(32))
    cuda_only(S.page_plan, good)
    for name, bad in (("new_tokens", i32(5)), ("block_table", i32(3, 8)), ("block_table", i32(32)), ("free_count", i32(2)),
                      ("free_list", i32(8, 8)), ("cu_tokens", i32(4)), ("positions", i32(31)), ("slot_map", i32(0)),
                      ("seqlens", i32(2, 2)), ("seqlens_out", i32(3)), ("free_count_out", i32(0)), ("err", i32(0))):
        refused(S.page_plan, good, name, bad)
    good = dict(page_size=16, seqlens=i32(4), finished=i32(4), block_table=i32(4, 8), free_list=i32(64), free_count=i32(1))
    cuda_only(S.page_release, good)
    for name, bad in (("finished", i32(3)), ("block_table", i32(5, 8)), ("free_count", i32(0)), ("seqlens_out", i32(5))):
        refused(S.page_release, good, name, bad)


# ---------------------------------------------------------------- norm + rotation
def rows(data=4096, st=128 * 4, sh=128):
    return S.RowsDesc(data, st, sh)


def qk(**kw):
    a = dict(num_tokens=8, num_q_heads=4, num_kv_heads=2, head_dim=128, rope_dim=128, dtype=0, rope_base=1e6, eps=1e-6)
    a.update(kw)
    return S.QkShape(**a)


def pool(**kw):
    a = dict(data=1 << 20, stride_page=2 * 16 * 128, stride_h=16 * 128, stride_t=128, num_pages=4, page_size=16)
    a.update(kw)
    return S.PoolDesc(**a)


def forward(shape=None, **kw):
    a = dict(q=rows(), k=rows(), v=None, wq=None, wk=None, pos=P, qo=rows(8192), ko=None, qn=None, kn=None, kc=None,
             vc=None, slots=None, live=None, err=None)
    a.update(kw)
    s = shape or qk()
    args = [ctypes.byref(x) if isinstance(x, ctypes.Structure) else x for x in a.values()]
    return lib.seer_qk_norm_rope(ctypes.byref(s), *args, None)


def test_norm_rope_refusals():
    for kw, st, word in ((dict(num_tokens=-1), 1, "num_tokens"), (dict(num_tokens=1 << 28), 2, "2^31"),
                         (dict(num_q_heads=0), 1, "heads"), (dict(head_dim=96), 2, "head_dim"),
                         (dict(rope_dim=24), 2, "rope_dim"), (dict(rope_dim=144), 2, "rope_dim"),
                         (dict(rope_dim=-16), 2, "rope_dim"), (dict(dtype=3), 2, "dtype"), (dict(rope_base=0), 1, "rope_base"),
                         (dict(rope_base=float("inf")), 1, "rope_base"), (dict(eps=-1), 1, "eps"),
                         (dict(eps=float("nan")), 1, "eps")):
        assert forward(qk(**kw)) == st and said(word), kw
    assert forward(qk(num_tokens=0), q=None) == 0
    assert forward(qo=None) == 1 and said("no output")
    assert forward(q=None) == 1 and said("q is NULL")
    assert forward(kn=rows(1 << 16), k=None) == 1 and said("k is NULL")
    assert forward(pos=None) == 1 and said("positions")
    assert forward(q=rows(4104)) == 1 and said("aligned")
    assert forward(q=rows(st=513)) == 1 and said("strides")
    assert forward(q=rows(sh=-128)) == 1 and said("strides")
    assert forward(qo=rows(8192, sh=64)) == 1 and said("overlap")
    assert forward(qo=rows(8192, st=0)) == 1 and said("overlap")
    assert forward(qn=rows(8192)) == 1 and said("share")
    assert forward(wq=ODD) == 1 and said("weight")
    assert forward(kc=pool()) == 1 and said("slot_map")
    assert forward(kc=pool(), slots=P, k=None) == 1 and said("k is NULL")
    assert forward(vc=pool(), slots=P) == 1 and said("v is NULL")
    assert forward(qk(dtype=2), kc=pool(), slots=P) == 2 and said("bf16 or fp16")
    assert forward(kc=pool(data=(1 << 20) + 8), slots=P) == 1 and said("aligned")
    assert forward(kc=pool(stride_t=64), slots=P) == 1 and said("strides")
    assert forward(kc=pool(num_pages=1 << 30), slots=P) == 2 and said("2^31")
    assert forward(kc=pool(), vc=pool(data=1 << 21, page_size=8), v=rows(), slots=P) == 1 and said("differ")
    assert forward(kc=pool(), vc=pool(), v=rows(), slots=P) == 1 and said("share")
    reaches_cuda(forward)


def backward(shape=None, **kw):
    a = dict(gq=rows(), gk=rows(1 << 16), gqn=None, gkn=None, q=rows(1 << 17), k=rows(1 << 18), wq=P, wk=P, pos=P,
             dq=rows(1 << 19), dk=rows(1 << 20), dwq=P, dwk=ctypes.c_void_p(8192), live=None, ws=P, n=1 << 23)
    a.update(kw)
    s = shape or qk()
    args = [ctypes.byref(x) if isinstance(x, ctypes.Structure) else x for x in a.values()]
    return lib.seer_qk_norm_rope_backward(ctypes.byref(s), *args, None)


def test_norm_rope_backward_refusals():
    n = lib.seer_qk_norm_rope_workspace_bytes(128)
    assert n == 8192 * 128 * 4 and lib.seer_qk_norm_rope_workspace_bytes(96) == 0
    assert backward(qk(head_dim=80)) == 2
    assert backward(dq=None, dk=None, wq=None, wk=None, dwq=None, dwk=None) == 1 and said("no output")
    assert backward(dq=None) == 1 and said("norm weight")
    assert backward(gq=None) == 1 and said("needs")
    assert backward(q=None) == 1 and said("q is NULL")
    assert backward(dwq=None) == 1 and said("together")
    assert backward(wk=None) == 1 and said("together")
    assert backward(wq=ODD) == 1 and said("weight")
    assert backward(dwq=ctypes.c_void_p(4098)) == 1 and said("gradient")
    assert backward(dk=rows(1 << 19)) == 1 and said("share")
    assert backward(dwk=P) == 1 and said("share")
    assert backward(dk=rows(1 << 20, sh=0)) == 1 and said("overlap")
    assert backward(pos=None) == 1 and said("positions")
    assert backward(ws=None) == 1 and said("workspace")
    assert backward(n=n - 1) == 1 and said("workspace")
    reaches_cuda(lambda: backward(n=n))


def test_norm_rope_binding_refusals():
    T, Hq, H, d = 8, 4, 2, 128
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)
    good = dict(q=z(T, Hq, d), k=z(T, H, d), positions=i32(T), q_out=z(T, Hq, d), k_out=z(T, H, d), q_weight=z(d),
                k_weight=z(d))
    cuda_only(S.qk_norm_rope, good)
    for name, bad in (("q", z(T, d)), ("q_out", z(T, H, d)), ("k_out", z(T - 1, H, d)), ("positions", None)):
        with pytest.raises((ValueError, TypeError)):
            S.qk_norm_rope(**{**good, name: bad})
    refused(S.qk_norm_rope, dict(good, q=None), "k", None)
    refused(S.qk_norm_rope, good, "q", z(T, Hq, d, dt=torch.float64), TypeError)
    refused(S.qk_norm_rope, good, "k_cache", z(4, H + 1, 16, d), (ValueError, TypeError))
    ws = torch.zeros(16, dtype=torch.uint8)
    back = dict(dq_out=z(T, Hq, d), dk_out=z(T, H, d), q=z(T, Hq, d), k=z(T, H, d), positions=i32(T), dq=z(T, Hq, d),
                dk=z(T, H, d), workspace=ws)
    cuda_only(S.qk_norm_rope_backward, back)
    refused(S.qk_norm_rope_backward, dict(back, q=None, dq=None), "k", z(T, d))


# ---------------------------------------------------------------- dense attention
def dense(kv=None, v=None, ws=P, n=1 << 40, q=P, lens=P, out=P, lse=None, **kw):
    a = dict(batch=4, num_q_heads=8, num_kv_heads=2, head_dim=128, dtype=0, page_size=16, window=0, softmax_scale=0.0)
    a.update(kw)
    s = S.DenseShape(**a)
    k = kv or contiguous()
    return lib.seer_dense_decode(ctypes.byref(s), q, ctypes.byref(k), ctypes.byref(v or k), lens, out, lse, ws, n, None, None)


def contiguous(**kw):
    a = dict(layout=0, data=4096, stride_b=2 * 64 * 128, stride_h=64 * 128, stride_t=128, num_tokens=64, num_pages=0,
             block_table=None, max_pages_per_seq=0)
    a.update(kw)
    return S.KVDesc(**a)


def test_dense_refusals():
    for kw, st, word in ((dict(batch=0), 1, "batch"), (dict(batch=4097), 2, "batch"), (dict(num_q_heads=9), 1, "multiple"),
                         (dict(num_q_heads=34), 2, "group"), (dict(head_dim=80), 2, "head_dim"), (dict(dtype=2), 2, "dtype"),
                         (dict(window=-1), 1, "window"), (dict(softmax_scale=-1.0), 1, "scale"),
                         (dict(softmax_scale=float("nan")), 1, "scale"), (dict(num_kv_heads=1 << 22, num_q_heads=1 << 22), 2, "2^24")):
        assert dense(**kw) == st and said(word), kw
    assert dense(contiguous(data=4104)) == 1 and said("aligned")
    assert dense(contiguous(stride_t=132)) == 1 and said("strides")
    assert dense(v=contiguous(stride_t=64)) == 1 and said("strides")
    assert dense(contiguous(num_tokens=0)) == 1
    assert dense(contiguous(layout=1)) == 1 and said("block_table")
    assert dense(contiguous(layout=2)) == 1 and said("layout")
    paged = contiguous(layout=1, block_table=4096, num_pages=8, max_pages_per_seq=4)
    assert dense(paged, page_size=0) == 1 and said("page_size")
    assert dense(contiguous(num_tokens=1 << 34)) == 2 and said("capacity")
    assert dense(contiguous(num_tokens=1 << 30), batch=64) == 2 and said("capacity")
    for name in ("q", "lens", "out", "ws"):
        assert dense(**{name: None}) == 1 and said("NULL")
    assert dense(q=ODD) == 1 and dense(out=ODD) == 1 and dense(ws=ODD) == 1
    assert dense(lse=ctypes.c_void_p(4098)) == 1
    reaches_cuda(dense)
    if torch.cuda.is_available():
        assert dense(n=16) == 1 and said("workspace")


def test_dense_binding_refusals():
    B, Hq, H, d = 2, 8, 2, 128
    half = torch.bfloat16
    z = lambda *s, dt=half: torch.zeros(*s, dtype=dt)

    def flat(t):
        return S.KVCache(S.KVDesc(0, 0, t.stride(0), t.stride(1), t.stride(2), t.shape[2], 0, None, 0), (t,), t.dtype)

    def paged(t, table):
        return S.KVCache(S.KVDesc(1, 0, t.stride(0), t.stride(1), t.stride(2), 0, t.shape[0], None, table.shape[1]),
                         (t, table), t.dtype)

    good = dict(q=z(B, Hq, d), k=flat(z(B, H, 64, d)), v=flat(z(B, H, 64, d)), seqlens=i32(B), out=z(B, Hq, d),
                workspace=torch.zeros(16, dtype=torch.uint8), lse=torch.zeros(B, Hq))
    cuda_only(S.dense_decode, good)
    cuda_only(S.dense_decode, dict(good, k=paged(z(9, H, 7, d), i32(B, 3))))
    for name, bad in (("q", z(B, d)), ("k", flat(z(B - 1, H, 64, d))), ("v", flat(z(B, H, 64, 64))),
                      ("v", flat(z(B, H + 1, 64, d))), ("k", paged(z(9, H, 7, d), i32(B - 1, 3))), ("seqlens", i32(B + 1)),
                      ("out", z(B, H, d)), ("lse", torch.zeros(B, H)), ("err", i32(0))):
        refused(S.dense_decode, good, name, bad)
    refused(S.dense_decode, dict(good, k=paged(z(9, H, 7, d), i32(B, 3))), "v", paged(z(9, H, 8, d), i32(B, 3)))
    refused(S.dense_decode, good, "v", flat(z(B, H, 64, d, dt=torch.float16)), TypeError)
    # the gated calls keep refusing caches of another type
    sh = S.Shape(B, Hq, H, d, 64, 64, 1)
    with pytest.raises(TypeError, match="bfloat16"):
        flat(z(B, H, 64, d, dt=torch.float16)).check(sh, "k")
