"""Refusals of the norm-and-rotate, append and chunk attention calls: the C ABI returns before
anything is launched, the binding raises before the C ABI is called (no GPU needed)."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import tiled_exact_attention_forward_b200 as fa
from tiled_exact_attention_forward_b200 import build as fa_build

P = ctypes.c_void_p
GOOD = P(0x100000)       # aligned, never dereferenced: validation fails first
MISALIGNED = P(0x100008)


@pytest.fixture(scope="module")
def lib():
    fa_build.build()
    return fa.library()


def strides(*v):
    return (ctypes.c_longlong * len(v))(*v)


ROWS = (4 * 10 * 128, 10 * 128, 128)  # [2, 4, 10, 128] contiguous


def norm_rope(lib, q=GOOD, k=GOOD, qo=GOOD, ko=GOOD, st=None, qw=None, kw=None, rope=GOOD, pos=None, pos_stride=0, B=2,
              Hq=4, Hk=4, N=10, d=128, rot=128, max_pos=10, eps=1e-6, inter=0, dtype=fa.FA_BF16, wdtype=fa.FA_BF16):
    st = strides(*ROWS * 4) if st is None else st
    return lib.fa_norm_rope(q, k, qo, ko, st, qw, kw, rope, pos, pos_stride, B, Hq, Hk, N, d, rot, max_pos, eps, inter,
                            dtype, wdtype, None)


@pytest.mark.parametrize("bad", [
    dict(q=None), dict(qo=None), dict(ko=None), dict(k=None), dict(q=MISALIGNED), dict(ko=MISALIGNED),
    dict(qw=MISALIGNED), dict(rope=MISALIGNED), dict(rope=None), dict(pos=P(0x100002)), dict(pos_stride=-1), dict(B=0),
    dict(Hq=0), dict(Hk=0), dict(N=0), dict(N=(1 << 30) + 1), dict(B=3, N=1 << 30), dict(rot=8), dict(rot=136), dict(rot=-16), dict(rot=0),
    dict(max_pos=0), dict(eps=float("nan")), dict(eps=float("inf")), dict(inter=2),
    dict(eps=-1.0, rot=0, rope=None),                                     # neither norm nor rotation
    dict(st=strides(*ROWS * 3, 4 * 10 * 128, 10 * 128, 127)),            # k_out's rows 254 bytes apart
    dict(st=strides(-5120, *(ROWS * 4)[1:])),
    dict(st=strides(*ROWS * 2, 5120, 0, 128, *ROWS)),                     # outputs on top of one another
])
def test_norm_rope_rejects(lib, bad):
    assert norm_rope(lib, **bad) == fa.FA_ERR_INVALID


@pytest.mark.parametrize("bad", [dict(d=96, rot=96), dict(dtype=7), dict(wdtype=fa.FA_FP16), dict(dtype=fa.FA_FP32)])
def test_norm_rope_has_no_kernel_for(lib, bad):
    assert norm_rope(lib, **bad) == fa.FA_ERR_UNSUPPORTED


def test_norm_rope_backward_rejects(lib):
    ws = lib.fa_norm_rope_backward_workspace_size(128)
    assert ws > 0 and ws % 256 == 0 and lib.fa_norm_rope_backward_workspace_size(96) == 0

    def bwd(q=GOOD, k=GOOD, gq=GOOD, gk=GOOD, dq=GOOD, dk=GOOD, dqw=GOOD, dkw=GOOD, eps=1e-6, ws_ptr=GOOD, ws_bytes=ws,
            st=None, d=128):
        return lib.fa_norm_rope_backward(q, k, gq, gk, dq, dk, strides(*ROWS * 6) if st is None else st, GOOD, GOOD, dqw,
                                         dkw, GOOD, None, 0, 2, 4, 4, 10, d, 64, 10, eps, 0, fa.FA_BF16, fa.FA_BF16,
                                         ws_ptr, ws_bytes, None)

    for bad in (dict(q=None), dict(k=None), dict(gq=None), dict(dq=None), dict(dk=None), dict(gk=None),
                dict(gk=None, dk=None),                                    # dk_weight without k
                dict(eps=-1.0),                                            # weight gradients without a norm
                dict(ws_ptr=None), dict(ws_ptr=P(0x100010)), dict(ws_bytes=ws - 1), dict(dqw=MISALIGNED),
                dict(gq=MISALIGNED), dict(st=strides(*ROWS * 5, 5120, 0, 128))):
        assert bwd(**bad) == fa.FA_ERR_INVALID, bad
    assert bwd(d=80) == fa.FA_ERR_UNSUPPORTED


def append(lib, k=GOOD, v=GOOD, q=GOOD, qo=GOOD, kp=GOOD, vp=GOOD, table=GOOD, cu=GOOD, lens=GOOD, qs=8 * 128, ks=256,
           vs=256, qw=None, kw=None, rope=GOOD, T=7, B=3, Hq=8, Hkv=2, num_blocks=10, bs=16, max_blocks=4, d=128, rot=128,
           max_pos=64, eps=1e-6, inter=0, dtype=fa.FA_BF16, wdtype=fa.FA_BF16):
    return lib.fa_append_paged(k, v, q, qo, kp, vp, table, cu, lens, qs, ks, vs, qw, kw, rope, T, B, Hq, Hkv, num_blocks,
                               bs, max_blocks, d, rot, max_pos, eps, inter, dtype, wdtype, None)


@pytest.mark.parametrize("bad", [
    dict(k=None), dict(v=None), dict(kp=None), dict(vp=None), dict(table=None), dict(lens=None), dict(q=None),
    dict(qo=None), dict(cu=None), dict(cu=P(0x100002)), dict(k=MISALIGNED), dict(vp=MISALIGNED), dict(kw=MISALIGNED),
    dict(T=0), dict(B=0), dict(Hkv=0), dict(Hq=0), dict(bs=24), dict(bs=8192), dict(num_blocks=0), dict(max_blocks=0),
    dict(max_blocks=1 << 28), dict(ks=248), dict(vs=260), dict(qs=1016), dict(rot=24), dict(rope=None), dict(max_pos=0),
    dict(eps=float("nan")), dict(inter=-1), dict(num_blocks=1 << 30),
])
def test_append_rejects(lib, bad):
    assert append(lib, **bad) == fa.FA_ERR_INVALID


@pytest.mark.parametrize("bad", [dict(d=64), dict(dtype=fa.FA_FP32, wdtype=fa.FA_FP32), dict(wdtype=fa.FA_FP16)])
def test_append_has_no_kernel_for(lib, bad):
    assert append(lib, **bad) == fa.FA_ERR_UNSUPPORTED


def extend(lib, q=GOOD, kp=GOOD, vp=GOOD, table=GOOD, cu=GOOD, lens=GOOD, o=GOOD, lse=None, qs=8 * 128, T=7, B=3, Hq=8,
           Hkv=2, num_blocks=10, bs=16, max_blocks=4, d=128, causal=1, window=0, dtype=fa.FA_BF16, ws=GOOD, ws_bytes=None):
    if ws_bytes is None:
        ws_bytes = lib.fa_extend_paged_workspace_size(7, 8, 2, 128)
    return lib.fa_extend_paged(q, kp, vp, table, cu, lens, o, lse, qs, T, B, Hq, Hkv, num_blocks, bs, max_blocks, d, 0.0,
                               causal, window, dtype, ws, ws_bytes, None)


@pytest.mark.parametrize("bad", [
    dict(q=None), dict(kp=None), dict(vp=None), dict(table=None), dict(lens=None), dict(o=None), dict(ws=None),
    dict(ws=P(0x100010)), dict(ws_bytes=100), dict(cu=None), dict(q=MISALIGNED), dict(o=MISALIGNED), dict(lse=P(0x100001)),
    dict(T=0), dict(B=0), dict(Hq=0), dict(Hkv=0), dict(Hq=7), dict(Hkv=3), dict(Hq=258), dict(bs=12), dict(bs=0),
    dict(bs=8192), dict(num_blocks=0), dict(max_blocks=0), dict(max_blocks=1 << 26), dict(causal=2), dict(window=-1),
    dict(window=(1 << 29) + 1), dict(qs=1020), dict(qs=512),
])
def test_extend_rejects(lib, bad):
    assert extend(lib, **bad) == fa.FA_ERR_INVALID


@pytest.mark.parametrize("bad", [dict(d=64), dict(dtype=fa.FA_FP32), dict(dtype=9)])
def test_extend_has_no_kernel_for(lib, bad):
    assert extend(lib, **bad) == fa.FA_ERR_UNSUPPORTED


def test_extend_workspace_size(lib):
    size = lib.fa_extend_paged_workspace_size
    assert size(1, 8, 2, 128) > 0 and size(1, 8, 2, 128) % 256 == 0
    assert size(1, 8, 2, 128) <= size(64, 8, 2, 128) <= size(5000, 8, 2, 128) == size(10 ** 6, 8, 2, 128)
    for bad in ((0, 8, 2, 128), (1, 8, 3, 128), (1, 0, 2, 128), (1, 300, 2, 128)):
        assert size(*bad) == 0


BF = torch.bfloat16


def test_binding_refuses_cpu_tensors():
    q = torch.zeros(1, 2, 8, 128, dtype=BF)
    pool, table, lens = torch.zeros(3, 2, 16, 128, dtype=BF), torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    for call in (lambda: fa.norm_rope(q, q), lambda: fa.norm_rope_backward(q, q, q, q),
                 lambda: fa.append_paged(q[0, :, :1].transpose(0, 1), q[0, :, :1].transpose(0, 1), pool, pool, table, lens),
                 lambda: fa.extend_paged(torch.zeros(1, 2, 128, dtype=BF), pool, pool, table, lens)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_unbound_module_refuses_calls():
    code = ("import torch; from tiled_exact_attention_forward_b200 import _calls\n"
            "try: _calls.norm_rope(*[None] * 10)\n"
            "except RuntimeError as e: assert 'not bound' in str(e)\n"
            "else: raise SystemExit(1)\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(fa.__file__)))
    assert subprocess.run([sys.executable, "-c", code], cwd=root).returncode == 0


def test_binding_refuses_what_is_no_tensor_or_number():
    q = torch.empty(1, 2, 8, 128, dtype=BF, device="meta")
    for call in (lambda: fa.norm_rope("q"), lambda: fa.norm_rope(None), lambda: fa.norm_rope(q, k=3),
                 lambda: fa.norm_rope(q, eps="1"), lambda: fa.norm_rope(q.double()),
                 lambda: fa.extend_paged(q[0], q, q, q, None), lambda: fa.append_paged(1, 2, 3, 4, 5, 6)):
        with pytest.raises(TypeError):
            call()


NOT_THE_DEVICE = r"^(?!.*CUDA)"


class TestBindingChecks:
    """Checks of shapes, types and layouts, which come before the device's: on tensors of the meta device."""

    @staticmethod
    def t(*shape, dtype=BF):
        return torch.empty(*shape, dtype=dtype, device="meta")

    @pytest.mark.parametrize("change", [
        dict(k=(1, 2, 9, 128)), dict(k=(2, 8, 128)), dict(k_dtype=torch.float16), dict(rope=(8, 130)), dict(rope=(8, 24)),
        dict(rope_dtype=torch.float64), dict(qw=(64,)), dict(qw_dtype=torch.float16), dict(eps=None), dict(eps=-1.0),
        dict(positions=(7,)), dict(positions=(8,), pos_dtype=torch.int64), dict(q_out=(1, 2, 8, 64)),
    ])
    def test_norm_rope(self, change):
        t = self.t
        with pytest.raises((ValueError, TypeError), match=NOT_THE_DEVICE):
            fa.norm_rope(t(1, 2, 8, 128), t(*change.get("k", (1, 2, 8, 128)), dtype=change.get("k_dtype", BF)),
                         t(*change.get("qw", (128,)), dtype=change.get("qw_dtype", BF)), None,
                         t(*change.get("rope", (8, 128)), dtype=change.get("rope_dtype", torch.float32)),
                         t(*change["positions"], dtype=change.get("pos_dtype", torch.int32)) if "positions" in change else None,
                         change.get("eps", 1e-6), q_out=t(*change["q_out"]) if "q_out" in change else None)

    def test_norm_rope_rows(self):
        with pytest.raises(ValueError, match="contiguous"):
            fa.norm_rope(self.t(1, 2, 128, 8).transpose(2, 3))
        with pytest.raises(ValueError, match="packed"):
            fa.norm_rope(self.t(8, 128))
        with pytest.raises(ValueError, match="go together"):
            fa.norm_rope_backward(self.t(1, 2, 8, 128), self.t(1, 2, 8, 128), self.t(1, 2, 8, 128), None)

    @pytest.mark.parametrize("change", [
        dict(k=(7, 3, 128)), dict(v=(6, 2, 128)), dict(vpool=(5, 2, 8, 128)), dict(table=(3,)), dict(lens=(4,)),
        dict(cu=(3,)), dict(no_cu=True), dict(lens_dtype=torch.int64), dict(q=(6, 8, 128)), dict(q=(7, 8, 64)),
        dict(k_dtype=torch.float16),
    ])
    def test_append(self, change):
        t, i32 = self.t, torch.int32
        with pytest.raises(ValueError, match=NOT_THE_DEVICE):
            fa.append_paged(t(*change.get("k", (7, 2, 128)), dtype=change.get("k_dtype", BF)), t(*change.get("v", (7, 2, 128))),
                            t(5, 2, 16, 128), t(*change.get("vpool", (5, 2, 16, 128))),
                            t(*change.get("table", (3, 4)), dtype=i32),
                            t(*change.get("lens", (3,)), dtype=change.get("lens_dtype", i32)),
                            None if "no_cu" in change else t(*change.get("cu", (4,)), dtype=i32),
                            q=t(*change["q"]) if "q" in change else None)

    @pytest.mark.parametrize("change", [
        dict(q=(7, 7, 128)), dict(q=(7, 8, 64)), dict(q=(7, 1024)), dict(out=(7, 8, 64)), dict(lse=(8, 7)), dict(cu=(3,)),
        dict(no_cu=True), dict(table=(3,)),
    ])
    def test_extend(self, change):
        t, i32 = self.t, torch.int32
        with pytest.raises(ValueError, match=NOT_THE_DEVICE):
            fa.extend_paged(t(*change.get("q", (7, 8, 128))), t(5, 2, 16, 128), t(5, 2, 16, 128),
                            t(*change.get("table", (3, 4)), dtype=i32), t(3, dtype=i32),
                            None if "no_cu" in change else t(*change.get("cu", (4,)), dtype=i32),
                            out=t(*change["out"]) if "out" in change else None,
                            lse=t(*change["lse"], dtype=torch.float32) if "lse" in change else None)

    def test_heads_apart(self):
        t, i32 = self.t, torch.int32
        q = t(7, 128, 8).transpose(1, 2)
        with pytest.raises(ValueError, match="heads"):
            fa.extend_paged(q, t(5, 2, 16, 128), t(5, 2, 16, 128), t(3, 4, dtype=i32), t(3, dtype=i32), t(4, dtype=i32))

    def test_window(self):
        t, i32 = self.t, torch.int32
        args = (t(7, 8, 128), t(5, 2, 16, 128), t(5, 2, 16, 128), t(3, 4, dtype=i32), t(3, dtype=i32), t(4, dtype=i32))
        for window in (-1, 2 ** 31, -2 ** 62):
            with pytest.raises(ValueError, match="window"):
                fa.extend_paged(*args, window=window)
        with pytest.raises((TypeError, OverflowError)):
            fa.extend_paged(*args, window=2 ** 70)
        with pytest.raises(ValueError, match="CUDA"):
            fa.extend_paged(*args, window=5)

    def test_workspace_of_fewer_bytes_than_elements(self):
        """An expanded or strided workspace would be written past its memory."""
        t, i32 = self.t, torch.int32
        q = t(1, 2, 8, 128)
        args = (t(7, 8, 128), t(5, 2, 16, 128), t(5, 2, 16, 128), t(3, 4, dtype=i32), t(3, dtype=i32), t(4, dtype=i32))
        u8 = torch.uint8
        for ws in (t(1, dtype=u8).expand(1 << 26), t(1 << 20, 128, dtype=u8)[:, :64], t(1 << 27, dtype=u8)[::2]):
            with pytest.raises(ValueError, match="workspace"):
                fa.norm_rope_backward(q, None, q, None, t(128), workspace=ws)
            with pytest.raises(ValueError, match="workspace"):
                fa.extend_paged(*args, workspace=ws)
        with pytest.raises(ValueError, match="CUDA"):
            fa.extend_paged(*args, workspace=t(1 << 26, dtype=u8))
