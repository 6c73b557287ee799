"""Host checks of the calls that make a step's inputs: bad arguments are refused before any
CUDA call, and good ones pass every check up to the device query."""
import ctypes

import pytest

from matrix_orthogonalising_optimizer_03_b200 import binding as B
from matrix_orthogonalising_optimizer_03_b200 import build as build_mod

FAKE = 1 << 40
GB = 1 << 30


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.load()


def act8(**kw):
    a = dict(X=FAKE, q=FAKE + GB, exps=FAKE + 2 * GB, rows=100, cols=70, ld_x=70, ld_q=80, ld_e=16, dtype=1,
             reserved=0)
    a.update(kw)
    return B.MuonAct8(**a)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), 3), (dict(rows=-1), 2), (dict(cols=0), 2), (dict(cols=(1 << 26) + 1, ld_x=1 << 27, ld_q=1 << 27), 2),
    (dict(ld_x=69), 2), (dict(ld_q=64), 2), (dict(ld_q=72), 2), (dict(ld_e=2), 2), (dict(ld_e=24), 2),
    (dict(X=None), 1), (dict(q=None), 1), (dict(exps=None), 1), (dict(X=FAKE + 1), 1), (dict(q=FAKE + GB + 8), 1),
    (dict(exps=FAKE + 2 * GB + 8), 1), (dict(dtype=0, X=FAKE + 2), 1), (dict(q=FAKE + 64), 4),
    (dict(exps=FAKE + 64), 4), (dict(rows=1 << 41), 2), (dict(rows=1 << 39, ld_x=1 << 30), 2)])
def test_act8_refusals(lib, kw, status):
    for f in (lib.muon_act8_store, lib.muon_act8_restore):
        arr = (B.MuonAct8 * 2)(act8(X=FAKE + 8 * GB, q=FAKE + 9 * GB, exps=FAKE + 10 * GB), act8(**kw))
        assert f(arr, 2, None) == status
    assert lib.muon_act8_store(None, 1, None) == 1 and lib.muon_act8_store(None, -1, None) == 1
    assert lib.muon_act8_store(None, 0, None) == 0 and lib.muon_act8_restore(None, 0, None) == 0


def test_act8_aliases_between_items(lib):
    two = (B.MuonAct8 * 2)(act8(), act8(X=FAKE + 8 * GB, exps=FAKE + 10 * GB))       # one q for both
    assert lib.muon_act8_store(two, 2, None) == 4
    shared = (B.MuonAct8 * 2)(act8(), act8(q=FAKE + 9 * GB, exps=FAKE + 10 * GB))    # one X for both
    assert lib.muon_act8_restore(shared, 2, None) == 4


def test_act8_read_buffers_may_be_shared(lib):
    """Shared activations of a store and shared checkpoints of a restore pass; whatever is written
    may not lie inside anything else, wherever it stands in a long list."""
    far = FAKE + 100 * GB

    def items(n, **last):
        return (B.MuonAct8 * n)(*(act8(X=FAKE, q=far + 2 * i * GB, exps=far + (2 * i + 1) * GB) for i in range(n - 1)),
                                act8(**last))
    for n in (3, 40):
        good = items(n)
        assert lib.muon_act8_store(good, n, None) not in (1, 2, 3, 4)
        assert lib.muon_act8_restore(good, n, None) == 4            # one X written n times
        inside = items(n, q=far + 64)                                # inside the first item's q
        assert lib.muon_act8_store(inside, n, None) == 4
        inside = items(n, X=far - 16, ld_x=1 << 20)                  # an X around other buffers
        assert lib.muon_act8_store(inside, n, None) == 4


class Strided:
    """What the binding looks at of a 2-D CUDA tensor (this machine may have none)."""
    is_cuda, device = True, "cuda:0"

    def __init__(self, rows, cols, ld, dtype, ptr=FAKE):
        self.shape, self.strides, self.dtype, self.ptr = (rows, cols), (ld, 1), dtype, ptr

    def dim(self):
        return 2

    def size(self, i):
        return self.shape[i]

    def stride(self, i):
        return self.strides[i]

    def data_ptr(self):
        return self.ptr


@pytest.mark.parametrize("ld,status", [(0, 2), (16, 2), (63, 2), (64, None), (80, None)])
def test_act8_rows_that_overlap_are_refused(lib, ld, status):
    """A broadcast row (stride 0) or overlapping windows reach the C call with the stride that they
    have, which refuses them; taken as dense they would be read and written past their end."""
    import torch
    ck = B.Act8(Strided(8, 64, 64, torch.int8, FAKE + GB), Strided(8, 16, 16, torch.uint8, FAKE + 2 * GB), 64)
    for dtype in (torch.float32, torch.bfloat16):
        arr = B._act8_array([Strided(8, 64, ld, dtype)], [ck])
        assert arr[0].ld_x == ld
        for f in (lib.muon_act8_store, lib.muon_act8_restore):
            got = f(arr, 1, None)
            assert got == status if status else got not in (1, 2, 3, 4)


@pytest.mark.parametrize("rows", [0, 1])
@pytest.mark.parametrize("ld", [0, 1, 64, 90])
def test_act8_a_single_row_may_have_any_stride(lib, rows, ld):
    import torch
    ck = B.Act8(Strided(rows, 64, ld, torch.int8, FAKE + GB), Strided(rows, 16, ld, torch.uint8, FAKE + 2 * GB), 64)
    arr = B._act8_array([Strided(rows, 64, ld, torch.float32)], [ck])
    assert lib.muon_act8_store(arr, 1, None) not in (1, 2, 3, 4)


def wgrad(**kw):
    a = dict(dY=FAKE, q=FAKE + GB, exps=FAKE + 2 * GB, dW=FAKE + 3 * GB, offsets=FAKE + 4 * GB, status_dev=None,
             tokens=100, out=50, in_=70, ld_dy=56, ld_q=80, ld_e=16, ld_w=70, stride_w=3500, groups=3, w_dtype=1,
             accumulate=0, reserved=0)
    a.update(kw)
    return B.MuonWeightGrad(**a)


@pytest.mark.parametrize("kw,status", [
    (dict(w_dtype=4), 3), (dict(tokens=-1), 2), (dict(out=0), 2), (dict(in_=0), 2), (dict(groups=0), 2),
    (dict(ld_dy=50), 2), (dict(ld_dy=48), 2), (dict(ld_q=64), 2), (dict(ld_q=72), 2), (dict(ld_e=8), 2),
    (dict(ld_w=69), 2), (dict(stride_w=3499), 2), (dict(accumulate=2), 1), (dict(dW=None), 1), (dict(offsets=None), 1),
    (dict(dY=None), 1), (dict(q=None), 1), (dict(exps=None), 1), (dict(dY=FAKE + 8), 1), (dict(q=FAKE + GB + 4), 1),
    (dict(exps=FAKE + 2 * GB + 4), 1), (dict(dW=FAKE + 3 * GB + 1), 1), (dict(offsets=FAKE + 4 * GB + 2), 1),
    (dict(status_dev=FAKE + 2), 1), (dict(dW=FAKE + 64), 4), (dict(dW=FAKE + GB + 64), 4),
    (dict(dW=FAKE + 2 * GB + 64), 4), (dict(dW=FAKE + 4 * GB), 4), (dict(status_dev=FAKE + 3 * GB + 400), 4),
    (dict(tokens=1 << 31), 2), (dict(tokens=(1 << 31) - 63), 2),
    (dict(out=1, in_=(1 << 31) - 500, ld_w=(1 << 31) - 1, ld_q=(1 << 31) - 16, ld_e=1 << 27, groups=1), 2),
    (dict(in_=1, out=(1 << 31) - 500, ld_dy=(1 << 31) - 8, groups=1), 2), (dict(out=1 << 20, in_=1 << 20, ld_w=1 << 20, ld_dy=1 << 20, ld_q=1 << 20,
                                     ld_e=1 << 20, groups=1), 2)])
def test_weight_grad_refusals(lib, kw, status):
    assert lib.muon_weight_grad(ctypes.byref(wgrad(**kw)), None, 0, None) == status
    assert lib.muon_weight_grad_workspace_size(ctypes.byref(wgrad(**kw))) == 0
    assert lib.muon_weight_grad(None, None, 0, None) == 1


def attention(**kw):
    a = B.MuonAttention()
    tok = dict(q=(0, 4), k=(1, 2), v=(2, 2), o=(3, 4), dout=(4, 4), dq=(5, 4), dk=(6, 2), dv=(7, 2))
    for n, (i, h) in tok.items():
        setattr(a, n, B.MuonHeads(FAKE + i * GB, h * 64, 64))
    a.lse, a.s_max, a.q_offsets, a.k_offsets = FAKE + 8 * GB, FAKE + 9 * GB, FAKE + 10 * GB, FAKE + 11 * GB
    a.q_tokens, a.k_tokens, a.n_seq, a.heads, a.kv_heads, a.head_dim = 100, 90, 3, 4, 2, 64
    a.causal, a.scale = 1, 0.125
    for n, v in kw.items():
        setattr(a, n, v)
    return a


FORWARD = [
    (dict(q_tokens=-1), 2), (dict(k_tokens=-1), 2), (dict(n_seq=0), 2), (dict(heads=0), 2), (dict(kv_heads=0), 2),
    (dict(heads=5), 2), (dict(head_dim=0), 2), (dict(head_dim=68), 2), (dict(head_dim=136), 2), (dict(causal=2), 1),
    (dict(scale=0.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(scale=-1.0), 1),
    (dict(q_offsets=None), 1), (dict(k_offsets=None), 1), (dict(q_offsets=FAKE + 10 * GB + 2), 1),
    (dict(lse=None), 1), (dict(lse=FAKE + 8 * GB + 2), 1), (dict(s_max=FAKE + 9 * GB + 1), 1),
    (dict(q=B.MuonHeads(None, 256, 64)), 1), (dict(v=B.MuonHeads(FAKE + 2 * GB + 8, 128, 64)), 1),
    (dict(q=B.MuonHeads(FAKE, 252, 64)), 2), (dict(q=B.MuonHeads(FAKE, 256, 60)), 2),
    (dict(q=B.MuonHeads(FAKE, 128, 64)), 2), (dict(k=B.MuonHeads(FAKE + GB, 128, 0)), 2),
    (dict(k=B.MuonHeads(FAKE + GB, 0, 64)), 2), (dict(o=B.MuonHeads(FAKE + 64, 256, 64)), 4),
    (dict(o=B.MuonHeads(FAKE, 256, 64)), 4), (dict(o=B.MuonHeads(FAKE + GB + 512, 256, 64)), 4),
    (dict(lse=FAKE), 4), (dict(lse=FAKE + 3 * GB), 4), (dict(s_max=FAKE + 8 * GB + 40), 4),
    (dict(s_max=FAKE + 2 * GB), 4), (dict(status_dev=FAKE + 10 * GB), 4), (dict(q_offsets=FAKE + 8 * GB), 4)]


@pytest.mark.parametrize("kw,status", FORWARD)
def test_attention_refusals(lib, kw, status):
    assert lib.muon_attention_forward(ctypes.byref(attention(**kw)), None) == status
    assert lib.muon_attention_forward(None, None) == 1


@pytest.mark.parametrize("n_seq", [1, 2, 3])
def test_attention_offsets_on_one_side(lib, n_seq):
    """A single sequence may have offsets of its rows or of its keys alone, or none; several need
    both. The workspace size is 0 for a refused call and launches nothing."""
    for q_off, k_off in ((None, FAKE + 11 * GB), (FAKE + 10 * GB, None), (None, None)):
        a = attention(n_seq=n_seq, q_offsets=q_off, k_offsets=k_off)
        assert (lib.muon_attention_workspace_size(ctypes.byref(a)) > 0) == (n_seq == 1)
        if n_seq > 1:
            assert lib.muon_attention_forward(ctypes.byref(a), None) == 1
            assert lib.muon_attention_backward(ctypes.byref(a), FAKE + 12 * GB, GB, None) == 1


@pytest.mark.parametrize("kw,status", [
    (dict(dout=B.MuonHeads(None, 256, 64)), 1), (dict(dq=B.MuonHeads(FAKE + 5 * GB, 264, 62)), 2),
    (dict(dq=B.MuonHeads(FAKE, 256, 64)), 4), (dict(dk=B.MuonHeads(FAKE + 7 * GB + 128, 128, 64)), 4),
    (dict(dv=B.MuonHeads(FAKE + 2 * GB, 128, 64)), 4), (dict(lse=FAKE + 5 * GB), 4), (dict(head_dim=4), 2),
    (dict(q_offsets=FAKE + 6 * GB), 4)])
def test_attention_backward_refusals(lib, kw, status):
    a = attention(**kw)
    assert lib.muon_attention_workspace_size(ctypes.byref(a)) == 0
    assert lib.muon_attention_backward(ctypes.byref(a), FAKE + 12 * GB, GB, None) == status
    assert lib.muon_attention_backward(None, None, 0, None) == 1


def test_attention_workspace(lib):
    a = attention()
    size = lib.muon_attention_workspace_size(ctypes.byref(a))
    assert size >= 4 * 4 * 100
    for ws, n in ((None, size), (FAKE + 12 * GB + 16, size), (FAKE + 12 * GB, size - 1)):
        assert lib.muon_attention_backward(ctypes.byref(a), ws, n, None) == 5


def test_interleaved_views_are_not_aliases(lib):
    """dq, dk and dv as views of one buffer, token-major and head-major. The workspace size is
    0 for a refused call and launches nothing."""
    def size(a):
        return lib.muon_attention_workspace_size(ctypes.byref(a))

    row, base = 8 * 64, FAKE + 5 * GB
    a = attention(dq=B.MuonHeads(base, row, 64), dk=B.MuonHeads(base + 512, row, 64),
                  dv=B.MuonHeads(base + 768, row, 64))
    assert size(a) > 0
    a.dv = B.MuonHeads(base + 768 - 16, row, 64)       # reaches into dk
    assert size(a) == 0
    a.dv = B.MuonHeads(base + 768, row + 8, 64)        # another token stride: may collide
    assert size(a) == 0
    # heads outermost: planes of 100 tokens
    a = attention(dq=B.MuonHeads(base, 64, 6400), dk=B.MuonHeads(base + 4 * 12800, 64, 6400),
                  dv=B.MuonHeads(base + 6 * 12800, 64, 6400), k_tokens=100)
    assert size(a) > 0
    a.dv = B.MuonHeads(base + 6 * 12800 - 16, 64, 6400)
    assert size(a) == 0


class Fake:
    """A contiguous CUDA tensor as the binding looks at it."""
    is_cuda, device = True, "cuda:0"

    def __init__(self, shape, dtype, i=0, device="cuda:0", dense=True):
        self.shape, self.dtype, self.i, self.device, self.dense = tuple(shape), dtype, i, device, dense
        self.is_cuda = device != "cpu"

    def dim(self):
        return len(self.shape)

    def size(self, i):
        return self.shape[i]

    def stride(self, i):
        n = 1
        for x in self.shape[i + 1:]:
            n *= x
        return n

    def numel(self):
        return self.stride(0) * self.shape[0]

    def unsqueeze(self, _):
        return Fake((1, *self.shape), self.dtype, self.i)

    def is_contiguous(self):
        return self.dense

    def data_ptr(self):
        return FAKE + self.i * GB


def test_workspaces_of_another_device_are_refused(lib):
    """A workspace on the CPU, on another GPU or with gaps raises before the call marshals it."""
    import torch
    hp, u8, bf = B.hparams(), torch.uint8, torch.bfloat16
    w, g, m = (Fake((64, 64), torch.float32, i) for i in range(3))
    ck = B.Act8(Fake((100, 64), torch.int8, 3), Fake((100, 16), u8, 4), 64)
    dy, dw = Fake((100, 64), bf, 5), Fake((64, 64), torch.float32, 6)
    x = [Fake((100, 2, 64), bf, 7 + i) for i in range(8)]
    lse = Fake((2, 100), torch.float32, 20)
    for ws in (Fake((1 << 28,), u8, 30, "cpu"), Fake((1 << 28,), u8, 30, "cuda:1"), Fake((1 << 28,), u8, 30, dense=False)):
        for call in (lambda: B.step_batched([w], [g], [m], hp, workspace=ws), lambda: B.Plan([w], [g], [m], hp, workspace=ws),
                     lambda: B.newton_schulz([w], [g], hp, workspace=ws),
                     lambda: B.WeightGradPlan(dy, ck, dw, workspace=ws),
                     lambda: B.AttentionPlan(*x[:4], lse, grads=x[4:], workspace=ws)):
            with pytest.raises(B.MuonError) as e:
                call()
            assert e.value.status == 5
    good = Fake((1 << 28,), u8, 30)
    assert B.AttentionPlan(*x[:4], lse, grads=x[4:], workspace=good).workspace is good


def test_sizes_match_c_compiler(tmp_path):
    import os
    import subprocess
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "muon.h"\nint main(void){printf("%zu %zu %zu %zu %zu\\n",'
                   'sizeof(muon_act8_t),sizeof(muon_weight_grad_t),sizeof(muon_attention_t),'
                   'offsetof(muon_attention_t, scale),offsetof(muon_weight_grad_t, accumulate));return 0;}\n')
    subprocess.run(["gcc", "-I", inc, str(src), "-o", str(tmp_path / "s")], check=True)
    got = list(map(int, subprocess.run([str(tmp_path / "s")], capture_output=True, text=True).stdout.split()))
    assert got == [ctypes.sizeof(B.MuonAct8), ctypes.sizeof(B.MuonWeightGrad), ctypes.sizeof(B.MuonAttention),
                   B.MuonAttention.scale.offset, B.MuonWeightGrad.accumulate.offset]


def test_binding_refuses_before_any_launch(lib):
    import torch
    t = torch.zeros(4, 4)
    for f in (lambda: B.new_act8(4, 4, device="cpu"), lambda: B.act8_store([t], []),
              lambda: B.weight_grad(t, None, t), lambda: B.weight_grad(t.to(torch.bfloat16), None, t),
              lambda: B.attention_forward(t, t, t),
              lambda: B.attention_forward(*(torch.zeros(4, 2, 8, dtype=torch.bfloat16),) * 3),
              lambda: B.attention_forward(*(torch.zeros(4, 2, 8),) * 3),
              lambda: B.Act8(t, t, 4)):
        with pytest.raises(B.MuonError):
            f()
