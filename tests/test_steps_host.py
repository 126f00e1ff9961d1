"""Refusals of the norm and the beam search that need no GPU: the C entry points'
checks before any device work, and the binding's checks of its tensors (stand-ins for
CUDA tensors, and entry points that record that they were reached)."""

import ctypes

import pytest
import torch

from tp_vocab_logits_gb300 import _build, hg

bf16, f32, i64 = torch.bfloat16, torch.float32, torch.int64


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return hg.load()


@pytest.mark.parametrize("args", [
    (0, 4, 0), (1 << 30, 4, 0), (64, 0, 0), (64, 1 << 30, 0), (64, 4, 3), (64, 4, -1)])
def test_norm_create_refuses(lib, args):
    out = ctypes.c_void_p(1)
    assert lib.hg_norm_create(*args, ctypes.byref(out)) == hg.HG_ERR_ARG
    assert out.value is None


@pytest.mark.parametrize("args", [
    (0, 4, 100, 4, 0),                       # no items
    (1, 0, 100, 4, 0), (1, hg.HG_MAX_BEAMS + 1, 100, 4, 0),
    (1, 4, 0, 4, 0), (1, 4, 1 << 30, 4, 0),  # vocabulary
    (1, 4, 100, 0, 0), (1, 4, 100, hg.HG_MAX_PICKS + 1, 0),
    (1, 2, 3, 7, 0),                         # more picks than candidates
    (1, 4, 100, 4, 3),                       # no such type of logits
    (1 << 29, 4, 100, 4, 0),                 # rows beyond int
])
def test_beam_create_refuses(lib, args):
    out = ctypes.c_void_p(1)
    assert lib.hg_beam_create(*args, ctypes.byref(out)) == hg.HG_ERR_ARG
    assert out.value is None


def test_calls_refuse_a_null_handle(lib):
    assert lib.hg_norm_create(64, 4, 0, None) == hg.HG_ERR_ARG
    assert lib.hg_beam_create(1, 4, 100, 4, 0, None) == hg.HG_ERR_ARG
    for kind in ("norm", "beam"):
        assert getattr(lib, f"hg_{kind}_destroy")(None) == hg.HG_OK
        assert getattr(lib, f"hg_{kind}_workspace_bytes")(None) == 0
    p = 4096
    assert lib.hg_norm_rows(None, p, 64, None, 0, None, 0, p, 1e-6, 1, p, 64, 0, None, 0, None,
                            None) == hg.HG_ERR_ARG
    assert lib.hg_norm_rows_grad(None, p, 64, p, p, p, 64, None, 0, 1, p, 64, None, 0,
                                 None) == hg.HG_ERR_ARG
    assert lib.hg_beam_select(None, p, 100, None, 1, p, None, -1, 1, p, p, 8, p, None,
                              None) == hg.HG_ERR_ARG
    assert lib.hg_beam_reorder(None, p, 8, 1, None, 0, None) == hg.HG_ERR_ARG


class Tensor:
    """What the binding asks of a CUDA tensor."""

    is_cuda = True

    def __init__(self, shape, dtype, device=1, strides=None):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device("cuda", device)
        self.strides = strides or torch.empty(self.shape, device="meta").stride()

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def stride(self, i=None):
        return self.strides if i is None else self.strides[i]

    def is_contiguous(self):
        return self.strides == torch.empty(self.shape, device="meta").stride()

    def data_ptr(self):
        return 4096

    def element_size(self):
        return self.dtype.itemsize

    def get_device(self):
        return self.device.index


STATE = ctypes.c_size_t * 7  # hg_beam_state


@pytest.fixture
def reached():
    """(name, arguments) of the entry points that calls reach."""
    _build.build()
    calls, keep = [], []
    mod = hg._step_call()
    vp, sz, i, f = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_float
    types = {"norm_rows": [vp, vp, sz, vp, sz, vp, sz, vp, f, i, vp, sz, i, vp, i, vp, vp],
             "norm_rows_grad": [vp, vp, sz, vp, vp, vp, sz, vp, sz, i, vp, sz, vp, i, vp],
             "beam_select": [vp, vp, sz, vp, sz, vp, vp, i, i, vp, vp, i, vp, vp, vp],
             "beam_reorder": [vp, vp, i, i, ctypes.POINTER(STATE), i, vp]}

    def entry(name):
        def record(*args):
            if name == "beam_reorder":
                args = args[:4] + ([tuple(args[4][k]) for k in range(args[5])],) + args[5:]
            calls.append((name, args))
            return hg.HG_OK
        keep.append(ctypes.CFUNCTYPE(ctypes.c_int, *types[name])(record))
        return ctypes.cast(keep[-1], ctypes.c_void_p).value

    mod.bind_steps(*[entry(n) for n in types], torch.int32, i64, f32, torch.float8_e4m3fn,
                   torch.bool, torch.uint8, lambda device: 0)
    yield calls
    hg._STEP_CALL = None  # bound to the library again by the next call


N, K = 3, 200
ITEMS, BEAMS, PICKS, V = 2, 3, 4, 50


def norm_handle():
    return hg.NormHandle(0, K, N, bf16, device=1)


def beam_handle():
    return hg.BeamHandle(0, ITEMS, BEAMS, V, PICKS, bf16, device=1)


def arguments(call):
    """The call's tensors by name, all on device 1."""
    def rows():
        return Tensor((N, K), bf16)

    def line():
        return Tensor((N,), f32)

    def out(dtype):
        return Tensor((ITEMS, PICKS), dtype)

    if call == "norm_rows":
        return {"x": rows(), "gain": Tensor((K,), bf16), "out": rows(), "residual": rows(),
                "sum_out": rows(), "rstd": line()}
    if call == "norm_rows_8":
        return {"x": rows(), "gain": Tensor((K,), bf16), "out": Tensor((N, K), torch.float8_e4m3fn),
                "scales": Tensor((N, 2), f32)}
    if call == "norm_rows_grad":
        return {"s": rows(), "gain": Tensor((K,), bf16), "rstd": line(), "grad_out": rows(),
                "grad_x": rows(), "grad_gain": Tensor((K,), bf16), "grad_sum": rows()}
    if call == "beam_select":
        return {"logits": Tensor((ITEMS * BEAMS, V), bf16), "scores": Tensor((ITEMS, BEAMS), f32),
                "tokens": out(i64), "parents": out(i64), "picked": out(f32),
                "lse": Tensor((ITEMS * BEAMS,), f32, strides=(4,)),
                "finished": Tensor((ITEMS, BEAMS), torch.bool),
                "picked_finished": out(torch.uint8)}
    return {"parents": Tensor((ITEMS, BEAMS), torch.int32),
            "states": [(Tensor((5, ITEMS * BEAMS, 7), bf16), 1), Tensor((ITEMS * BEAMS, 9), f32)]}


def make(call, args):
    if call == "beam_select":
        hg.hg_beam_select(beam_handle(), end=5, **args)
    elif call == "beam_reorder":
        hg.hg_beam_reorder(beam_handle(), **args)
    elif call == "norm_rows_grad":
        hg.hg_norm_rows_grad(norm_handle(), **args)
    else:
        hg.hg_norm_rows(norm_handle(), **args)


CALLS = ("norm_rows", "norm_rows_8", "norm_rows_grad", "beam_select", "beam_reorder")


@pytest.mark.parametrize("call", CALLS)
def test_tensors_of_the_handles_device_are_served(reached, call):
    make(call, arguments(call))
    assert [c[0] for c in reached] == [call.removesuffix("_8")]


@pytest.mark.parametrize("call,name", [(c, n) for c in CALLS for n in arguments(c)])
def test_a_tensor_of_another_device_is_refused(reached, call, name):
    args = arguments(call)
    t = args[name][0][0] if name == "states" else args[name]
    t.device = torch.device("cuda", 0)
    with pytest.raises(ValueError, match=f"{name}: need a tensor on cuda:1, got one on cuda:0"):
        make(call, args)
    assert reached == []


@pytest.mark.parametrize("call,name", [(c, n) for c in CALLS for n in arguments(c)
                                       if n != "states"])
@pytest.mark.parametrize("how", ["type", "shape", "gap"])
def test_another_type_or_shape_is_refused(reached, call, name, how):
    """A gap between the elements of a row or line is refused, but in lse."""
    args = arguments(call)
    t = args[name]
    if how == "type":
        args[name] = Tensor(t.shape, torch.float64)
    elif how == "shape":
        args[name] = Tensor((*t.shape[:-1], t.shape[-1] + 1), t.dtype)
    elif name == "lse":
        return
    else:
        args[name] = Tensor(t.shape, t.dtype, strides=tuple(2 * s for s in t.stride()))
    with pytest.raises(ValueError, match=":"):
        make(call, args)
    assert reached == []


def test_row_strides_reach_the_library(reached):
    args = arguments("norm_rows")
    args["residual"] = Tensor((N, K), bf16, strides=(K + 8, 1))
    make("norm_rows", args)
    assert reached[0][1][2] == K and reached[0][1][4] == K + 8
    args["residual"] = Tensor((N, K), bf16, strides=(K - 1, 1))
    with pytest.raises(ValueError, match="residual: rows overlap"):
        make("norm_rows", args)
    args = arguments("beam_select")
    args["logits"] = Tensor((ITEMS * BEAMS, V), bf16, strides=(V + 3, 1))
    make("beam_select", args)
    assert reached[1][1][2] == V + 3 and reached[1][1][4] == 4
    for call, name in (("beam_select", "logits"), ("norm_rows", "x"), ("norm_rows_grad", "s")):
        args = arguments(call)
        args[name] = Tensor((4,), bf16)
        with pytest.raises(ValueError, match=f"{name}:"):
            make(call, args)


def test_scale_blocks(reached):
    args = arguments("norm_rows_8")
    make("norm_rows_8", args)
    args["scales"] = Tensor((N, 1), f32)
    make("norm_rows_8", args)
    assert [c[1][12] for c in reached] == [3, 3] and [c[1][14] for c in reached] == [128, 0]
    args["out"] = Tensor((N, K), bf16)
    with pytest.raises(ValueError, match="out: need a CUDA tensor of torch.float8_e4m3fn"):
        make("norm_rows_8", args)
    del args["scales"]
    make("norm_rows_8", args)
    assert reached[2][1][12] == 0


@pytest.mark.parametrize("end", [-2, V, 1 << 40])
def test_an_end_outside_the_vocabulary_is_refused(reached, end):
    with pytest.raises(ValueError, match="end:"):
        hg.hg_beam_select(beam_handle(), end=end, **arguments("beam_select"))
    assert reached == []


R = ITEMS * BEAMS


@pytest.mark.parametrize("state,want", [
    # outer, its stride, row stride, pieces, their stride, bytes of a run
    (Tensor((R, 9), f32), (1, 0, 36, 1, 0, 36)),
    (Tensor((R,), i64), (1, 0, 8, 1, 0, 8)),
    ((Tensor((5, R, 7), bf16), 1), (1, 0, 14, 5, R * 14, 14)),
    ((Tensor((5, R, 7), bf16), -2), (1, 0, 14, 5, R * 14, 14)),
    # layers, rows, heads, 3 of 10 positions, width
    ((Tensor((5, R, 2, 3, 8), bf16, strides=(R * 160, 160, 80, 8, 1)), 1),
     (5, R * 320, 320, 2, 160, 48)),
    # rows first: layers and heads are one step
    (Tensor((R, 5, 2, 3, 8), bf16, strides=(800, 160, 80, 8, 1)), (1, 0, 1600, 10, 160, 48)),
    # dimensions in another order than their strides
    ((Tensor((8, R, 3), bf16, strides=(1, 24, 8)), 1), (1, 0, 48, 1, 0, 48)),
    # no contiguous run: single elements
    (Tensor((R, 4), f32, strides=(8, 2)), (1, 0, 32, 4, 8, 4)),
    (Tensor((R, 1, 1), f32), (1, 0, 4, 1, 0, 4)),
])
def test_states_as_runs(reached, state, want):
    hg.hg_beam_reorder(beam_handle(), Tensor((ITEMS, BEAMS), i64), [state])
    name, args = reached[0]
    assert args[2:4] == (8, ITEMS) and args[4][0] == (4096, *want)


@pytest.mark.parametrize("states,match", [
    ([Tensor((R + 1, 4), f32)], "rows in dimension 0"),
    ([(Tensor((4, R), f32), 2)], "rows in dimension 2"),
    ([(Tensor((4, R), f32), "1")], "pairs"),
    ([(Tensor((R, 4), f32),)], "pairs"),
    ([7], "pairs"),
    ([Tensor((R, 2, 3, 4, 5), f32, strides=(9000, 2000, 500, 100, 1))], "more than two steps"),
    (Tensor((R, 4), f32), "list"),
    ([Tensor((R, 4), f32)] * (hg.HG_MAX_STATES + 1), "at most"),
])
def test_states_that_are_refused(reached, states, match):
    good = Tensor((R, 4), f32)
    if isinstance(states, list):
        states = [good] + states
    with pytest.raises(ValueError, match=match):
        hg.hg_beam_reorder(beam_handle(), Tensor((ITEMS, BEAMS), i64), states)
    assert reached == []


def test_create_names_the_type():
    with pytest.raises(ValueError, match="dtype"):
        hg.hg_norm_create(64, 4, dtype=torch.float64)
    with pytest.raises(ValueError, match="dtype"):
        hg.hg_beam_create(1, 4, 100, 4, dtype=torch.float8_e4m3fn)
