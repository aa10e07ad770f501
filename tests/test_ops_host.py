"""Host-side checks of the operators beside the layer (include/hq_ops.h), no
GPU needed: every refusal of the C ABI happens before the device is touched,
and the Python binding refuses tensors that do not fit."""
import ctypes

import pytest

FAKE = 0x10000      # aligned, never dereferenced: every call below is refused or a no-op
FAR = 0x100000000   # a second buffer far from FAKE
OK, INVALID, UNSUPPORTED, MISALIGNED = 0, 1, 2, 3


@pytest.fixture(scope="module")
def hq():
    from hadamard_rotated_bit_token_b200 import build as hq_build
    hq_build.build()
    import hadamard_rotated_bit_token_b200 as hq_mod
    hq_mod.load_library()
    return hq_mod


def _ep(hq, act=0, residual=None, gate=None, gate_rows=0):
    e = hq.Epilogue(act)
    e._residual, e._gate, e.gate_rows = residual, gate, gate_rows
    return ctypes.byref(e)


def test_dense_refusals(hq):
    lib = hq.load_library()

    def call(K=64, N=64, T=4, X=FAKE, W=2 * FAR, b=None, ep=None, Y=FAR, desc=True):
        d = ctypes.byref(hq.DenseDesc(K, N)) if desc else None
        return lib.hq_dense(d, X, T, W, b, ep, Y, None)

    assert call(desc=False) == INVALID
    assert call(K=0) == INVALID and call(N=-8) == INVALID and call(T=-1) == INVALID
    assert call(K=60) == UNSUPPORTED and call(N=20) == UNSUPPORTED
    assert call(K=(1 << 20) + 8) == UNSUPPORTED and call(T=2 ** 31 - 255) == UNSUPPORTED
    for name in ("X", "W", "Y"):
        assert call(**{name: None}) == INVALID
        assert call(**{name: FAKE + 8}) == MISALIGNED
    assert call(b=FAKE + 4) == MISALIGNED
    # Y over an input
    assert call(Y=FAKE) == INVALID
    assert call(Y=FAKE + 64 * 2) == INVALID
    assert call(Y=2 * FAR - 16) == INVALID
    assert call(b=FAR + 16) == INVALID
    # the epilogue
    assert call(ep=_ep(hq, act=5)) == INVALID and call(ep=_ep(hq, act=-1)) == INVALID
    assert call(ep=_ep(hq, gate=3 * FAR)) == INVALID               # gate_rows 0
    assert call(ep=_ep(hq, gate=3 * FAR, gate_rows=-2)) == INVALID
    assert call(ep=_ep(hq, residual=3 * FAR + 8)) == MISALIGNED
    assert call(ep=_ep(hq, gate=3 * FAR + 2, gate_rows=1)) == MISALIGNED
    assert call(ep=_ep(hq, residual=FAR + 128)) == INVALID         # partly Y
    assert call(ep=_ep(hq, gate=FAR + 16, gate_rows=4)) == INVALID  # the gate inside Y
    # nothing to do: no pointer is looked at, but the description is
    assert call(T=0, X=None, W=None, Y=None) == OK
    assert call(T=0, ep=_ep(hq, act=9)) == INVALID


def test_linear_ep_refusals(hq):
    lib = hq.load_library()
    D = hq.LayerDesc

    def call(desc, T=8, a=FAKE, sx=FAKE, m=None, w=FAKE, sw=FAKE, cs=None, b=None, ep=None, y=FAR):
        return lib.hq_linear_ep(None if desc is None else ctypes.byref(desc), T, a, sx, m, w, sw,
                                cs, b, ep, y, None, None)

    d = D(1024, 64, 1024)
    assert call(None) == INVALID and call(d, T=-1) == INVALID and call(d, a=None) == INVALID
    assert call(D(1000, 64, 8)) == UNSUPPORTED and call(D(1024, 24, 1024)) == UNSUPPORTED
    assert call(d, y=FAR + 2) == MISALIGNED and call(d, m=FAKE) == INVALID
    assert call(d, ep=_ep(hq, act=7)) == INVALID
    assert call(d, ep=_ep(hq, gate=3 * FAR)) == INVALID
    assert call(d, ep=_ep(hq, residual=FAR + 64)) == INVALID
    assert call(d, ep=_ep(hq, residual=3 * FAR + 4)) == MISALIGNED
    assert call(d, T=2 ** 31 - 255, ep=_ep(hq, act=1)) == UNSUPPORTED
    assert call(d, T=0, a=None, ep=_ep(hq, act=1)) == OK


def test_group_norm_refusals(hq):
    lib = hq.load_library()

    def call(C=64, G=8, act=0, eps=1e-5, B=2, S=16, X=FAKE, ga=None, be=None, Y=FAR, ws=None,
             nws=0, desc=True):
        d = ctypes.byref(hq.GroupNormDesc(C, G, act, eps)) if desc else None
        return lib.hq_group_norm(d, X, B, S, ga, be, Y, ws, nws, None)

    assert call(desc=False) == INVALID
    assert call(C=0) == INVALID and call(G=0) == INVALID and call(act=5) == INVALID
    assert call(eps=-1.0) == INVALID and call(eps=float("nan")) == INVALID
    assert call(eps=float("inf")) == INVALID
    assert call(G=7) == UNSUPPORTED and call(C=8200, G=8) == UNSUPPORTED
    assert call(B=-1) == INVALID and call(S=-1) == INVALID
    assert call(X=None) == INVALID and call(Y=None) == INVALID
    assert call(X=FAKE + 2) == MISALIGNED and call(Y=FAR + 8) == MISALIGNED
    assert call(ga=FAKE + 2) == MISALIGNED and call(be=FAKE + 4) == MISALIGNED
    assert call(Y=FAKE + 16) == INVALID and call(X=FAR - 32) == INVALID
    assert call(ga=FAR + 16) == INVALID and call(be=FAR + 32) == INVALID
    assert call(B=2 ** 31) == UNSUPPORTED and call(S=2 ** 31) == UNSUPPORTED
    assert call(B=0, X=None, Y=None) == OK and call(S=0, X=None) == OK
    assert lib.hq_group_norm_workspace_bytes(None, 1, 1) == 0
    assert hq.hq_group_norm_workspace_bytes(hq.GroupNormDesc(64, 7), 1, 1) == 0
    assert hq.hq_group_norm_workspace_bytes(hq.GroupNormDesc(64, 8), 0, 5) == 0


def test_binding_refusals(hq):
    torch = pytest.importorskip("torch")
    t = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device memory"):
        hq.hq_dense(hq.DenseDesc(64, 64), t, t, None, None, t)
    with pytest.raises(ValueError, match="device memory"):
        hq.hq_group_norm(hq.GroupNormDesc(64, 8), t, None, None, t)
    with pytest.raises(ValueError, match="shape"):
        hq.hq_group_norm(hq.GroupNormDesc(32, 8), t, None, None, t)
    with pytest.raises(ValueError, match="device memory"):
        hq.hq_linear_ep(hq.LayerDesc(64, 64, 64), t, None, None, t, t, t, t, None, t)
    with pytest.raises(ValueError, match="gate_rows"):
        hq.Epilogue(0, gate=t)
    with pytest.raises(ValueError, match="device memory"):
        hq.Epilogue(0, residual=t)


def test_block_refusals(hq):
    class Layer:
        desc = hq.LayerDesc(64, 32, 64)
    norm = hq.GroupNorm(64, 8)
    with pytest.raises(ValueError, match="channels"):
        hq.PointwiseBlock(hq.GroupNorm(32, 8), Layer())
    with pytest.raises(ValueError, match="outputs"):
        hq.PointwiseBlock(norm, Layer(), residual=True)
    with pytest.raises(ValueError, match="HadamardQuantLinear"):
        hq.PointwiseBlock(norm, Layer(), act=hq.HQ_ACT_SILU)


def test_sizes_past_the_coordinates_are_refused(hq):
    lib = hq.load_library()
    d = hq.DenseDesc(8, 2 ** 30 + 8)
    assert lib.hq_dense(ctypes.byref(d), FAKE, 1, 64 * FAR, None, None, FAR, None) == UNSUPPORTED
    d = hq.LayerDesc(16, 2 ** 30 + 16, 16)
    assert lib.hq_linear_ep(ctypes.byref(d), 1, FAKE, 2 * FAKE, None, 64 * FAR, 3 * FAR, None, None,
                            None, 5 * FAR, None, None) == UNSUPPORTED


class _OnDevice:
    """A stand-in for a CUDA tensor: what the binding asks of one, no memory."""

    def __init__(self, address, shape, dtype):
        self._address, self.shape, self.dtype, self.is_cuda = address, shape, dtype, True

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self._address


def test_a_reused_epilogue_forgets_tensors_taken_away(hq):
    """An Epilogue whose residual or gate is set to None after a call passes no
    address of the old one on, and one that is exchanged passes the new one."""
    torch = pytest.importorskip("torch")
    bf16 = torch.bfloat16
    rt = type("Runtime", (), {"bf16": bf16})
    ep = hq.Epilogue(hq.HQ_ACT_SILU, _OnDevice(FAKE, (4, 64), bf16), _OnDevice(FAR, (2, 64), bf16), 2)
    hq._epilogue_ref(rt, ep, 4, 64, 0)
    assert (ep._residual, ep._gate) == (FAKE, FAR)
    ep.residual = None
    hq._epilogue_ref(rt, ep, 4, 64, 0)
    assert (ep._residual, ep._gate) == (None, FAR)
    ep.gate = _OnDevice(2 * FAR, (2, 64), bf16)
    hq._epilogue_ref(rt, ep, 4, 64, 0)
    assert (ep._residual, ep._gate) == (None, 2 * FAR)
    ep.gate = None
    hq._epilogue_ref(rt, ep, 4, 64, 0)
    assert (ep._residual, ep._gate) == (None, None)


def test_known_faults_only(hq):
    lib = hq.load_library()
    for kind in (hq.HQ_FAULT_SPLITK_WITHHOLD_STAGE, hq.HQ_FAULT_TILE_WITHHOLD_STAGE,
                 hq.HQ_FAULT_TILE_WITHHOLD_RESIDUAL):
        assert lib.hq_debug_inject_fault(kind) == OK
    assert lib.hq_debug_inject_fault(hq.HQ_FAULT_NONE) == OK
    assert lib.hq_debug_inject_fault(-1) == INVALID and lib.hq_debug_inject_fault(100) == INVALID


def _bare_layer(hq):
    """A layer with weights of no use, in host memory: its bookkeeping alone."""
    torch = pytest.importorskip("torch")
    lay = hq.HadamardQuantLinear.__new__(hq.HadamardQuantLinear)
    lay.desc = hq.LayerDesc(64, 32, 16, act_gran=hq.HQ_PER_TENSOR_DYNAMIC)
    lay.w_codes = torch.zeros((32, 64), dtype=torch.int8)
    lay.workspace = torch.empty(16, dtype=torch.uint8)
    lay._bufs = {}
    return lay


def test_activation_buffers_of_two_streams_share_no_memory(hq):
    """Calls with the same number of tokens on two streams may run at once: each
    stream has codes, scale, mean and workspace of its own, found again."""
    lay, stream = _bare_layer(hq), [1]
    lay._stream_key = lambda: stream[0]
    one = lay.buffers(5)
    stream[0] = 2
    two = lay.buffers(5)
    for name in ("a_codes", "a_scale", "a_mean", "workspace"):
        assert one[name].data_ptr() != two[name].data_ptr(), name
    assert lay.buffers(5) is two
    stream[0] = 1
    assert lay.buffers(5) is one and lay.buffers(6) is not one


def test_activation_buffers_of_many_token_counts_are_bounded(hq):
    """What forward takes for itself is given back after other token counts; what
    a caller asked for stays."""
    lay = _bare_layer(hq)
    asked = lay.buffers(1000)
    for T in range(1, 100):
        lay._set_for(T, False)
    assert len(lay._bufs) == lay.KEPT_SETS + 1
    last = lay._set_for(99, False)
    assert lay.buffers(99) is last and lay.buffers(1000) is asked


def test_a_layers_launches_all_go_to_its_own_device(hq, monkeypatch):
    """A layer on device 1 called while device 0 is current: the quantizer and the
    product both run with device 1 current, and device 0 is current again after."""
    torch = pytest.importorskip("torch")
    current, seen = [0], []

    class Guard:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            self.old, current[0] = current[0], self.dev

        def __exit__(self, *exc):
            current[0] = self.old

    rt = type("Runtime", (), dict(
        current_device=staticmethod(lambda: current[0]), device_guard=Guard,
        stream_of=staticmethod(lambda dev: 100 + dev), capturing=staticmethod(lambda: False)))
    monkeypatch.setattr(hq, "_rt", rt)
    for name in ("hq_quantize_act", "hq_linear", "hq_linear_ep", "hq_gw_quantize_act",
                 "hq_gw_linear"):
        monkeypatch.setattr(hq, name, lambda *a, _n=name, **k: seen.append((_n, current[0])))

    class On1(_OnDevice):
        device = "cuda:1"

        def get_device(self):
            return 1

    X = On1(FAKE, (4, 64), torch.bfloat16)
    lay = _bare_layer(hq)
    lay.use_sigma, lay.w_scale, lay.colsum, lay.bias_f32 = False, None, None, None
    gw = hq.GroupWiseQuantLinear.__new__(hq.GroupWiseQuantLinear)
    gw.desc, gw._bufs, gw.use_sigma = hq.GwDesc(64, 32, 64, 0), {}, False
    gw.l1s = gw.l2b = gw.w_scale = gw.bias_f32 = None
    for layer in (lay, gw):
        layer.w_codes = On1(FAR, (32, 64), torch.int8)
        layer._new_buffers = lambda T: dict.fromkeys(
            ("a_codes", "a_scale", "a_mean", "u", "workspace"))
    Y = On1(2 * FAR, (4, 32), torch.bfloat16)
    lay.forward(X, Y)
    lay.forward(X, Y, epilogue=hq.Epilogue(hq.HQ_ACT_SILU))
    gw.forward(X, Y)
    assert seen == [("hq_quantize_act", 1), ("hq_linear", 1), ("hq_quantize_act", 1),
                    ("hq_linear_ep", 1), ("hq_gw_quantize_act", 1), ("hq_gw_linear", 1)]
    assert current == [0] and all(key == (4, 101) for key in lay._bufs)
    # an input on another device than the layer's is refused
    for layer in (lay, gw):
        with pytest.raises(ValueError, match="device"):
            layer.forward(torch.zeros(4, 64, dtype=torch.bfloat16), Y)


def test_group_norm_remembers_a_bounded_number_of_sizes(hq, monkeypatch):
    """A norm called with a new image size every time does not grow."""
    torch = pytest.importorskip("torch")
    import contextlib
    monkeypatch.setattr(hq, "_rt", type("Runtime", (), dict(
        device_guard=staticmethod(lambda dev: contextlib.nullcontext()), u8=torch.uint8)))
    asked = []
    monkeypatch.setattr(hq, "hq_group_norm", lambda *a: asked.append(a[-1]))

    class Input(_OnDevice):
        def numel(self):
            n = 1
            for k in self.shape:
                n *= k
            return n

        def new_empty(self, n, dtype=None):
            return ("workspace", n)

    norm = hq.GroupNorm(64, 8)
    for S in range(20000, 21000):
        X = Input(FAKE, (1, S, 64), torch.bfloat16)
        norm(X, X)
    assert len(norm._ws_bytes) <= 64 and len(asked) == 1000
    want = hq.hq_group_norm_workspace_bytes(norm.desc, 1, 20999)
    assert want > 0 and asked[-1] == ("workspace", want)


def test_an_epilogue_shared_by_two_threads_never_loses_its_gate(hq):
    """A call refreshes the addresses of its epilogue; another thread's call may be
    reading them, so neither is ever seen without the tensor it has."""
    torch = pytest.importorskip("torch")
    written = []

    class Watched(hq.Epilogue):
        def __setattr__(self, name, value):
            written.append((name, value))
            super().__setattr__(name, value)

    bf16 = torch.bfloat16
    ep = Watched(0, _OnDevice(FAKE, (4, 64), bf16), _OnDevice(FAR, (2, 64), bf16), 2)
    written.clear()
    hq._epilogue_ref(type("Runtime", (), {"bf16": bf16}), ep, 4, 64, 0)
    assert sorted(written) == [("_gate", FAR), ("_residual", FAKE)]
