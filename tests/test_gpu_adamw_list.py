"""GPU tests of the AdamW list on streams other than the current one: the
results are those of the same steps on one stream, bit for bit."""
import pytest
import torch

import token_dispatch_grouped_top_amd as mok

pytestmark = pytest.mark.gpu
HYPER = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, seed=3)
SIZES = (5000, 33, 4096, 1)


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def _tensors():
    """Tensors of both state formats, the same on each call."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    out = []
    for i, n in enumerate(SIZES):
        t = dict(p=torch.randn(n, generator=gen, device="cuda"))
        if i % 2:
            t.update({s: torch.zeros(n, dtype=torch.uint8, device="cuda") for s in ("m", "v")})
            t.update({s: torch.zeros((n + 31) // 32, dtype=torch.uint8, device="cuda") for s in ("m_scale", "v_scale")})
        else:
            t.update(m=torch.zeros(n, device="cuda"), v=torch.zeros(n, device="cuda"))
        out.append(t)
    return out


def _gradients(step):
    gen = torch.Generator(device="cuda").manual_seed(100 + step)
    return [torch.randn(n, generator=gen, device="cuda") for n in SIZES]


def _with(ts, grads):
    return [dict(t, grad=g) for t, g in zip(ts, grads)]


def _equal(a, b):
    return all(torch.equal(x[k], y[k]) for x, y in zip(a, b) for k in x)


def _plain(steps):
    ts = _tensors()
    for step in range(1, steps + 1):
        mok.mok_adamw_step(mok.AdamwTensors(_with(ts, _gradients(step))), step=step, **HYPER)
    torch.cuda.synchronize()
    return ts


@pytest.mark.parametrize("how", ["object", "handle", "current"])
@pytest.mark.parametrize("build_here", [False, True])
def test_new_lists_on_a_side_stream(how, build_here):
    """New gradients and a new list for each step, the list dropped while its step runs on a side stream that waits for
    the current one."""
    want, ts = _plain(4), _tensors()
    side = torch.cuda.Stream()
    argument = side.cuda_stream if how == "handle" else side
    for step in range(1, 5):
        grads = _gradients(step)
        if how == "current":
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                mok.mok_adamw_step(mok.AdamwTensors(_with(ts, grads)), step=step, **HYPER)
            for g in grads:
                g.record_stream(side)             # the gradients are memory of a stream that was not current
        else:
            lst = mok.AdamwTensors(_with(ts, grads), stream=None if build_here else argument)
            side.wait_stream(torch.cuda.current_stream())
            mok.mok_adamw_step(lst, step=step, stream=argument, **HYPER)
            del lst
        del grads
        torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert _equal(want, ts)


def test_list_built_on_a_side_stream_and_used_on_the_current_one():
    want, ts = _plain(1), _tensors()
    side = torch.cuda.Stream()
    lst = mok.AdamwTensors(_with(ts, _gradients(1)), stream=side)
    mok.mok_adamw_step(lst, step=1, **HYPER)
    torch.cuda.synchronize()
    assert _equal(want, ts)


def test_list_built_inside_a_capture():
    """The graph writes the table anew on each replay; beside a capture, on a stream that is not captured, it is refused."""
    ts, grads = _tensors(), _gradients(1)
    scalars = torch.zeros(4, device="cuda")
    scalars[0], scalars[1] = HYPER["lr"], 1.0
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lst = mok.AdamwTensors(_with(ts, grads))
        mok.mok_adamw_step(lst, step=1, scalars=scalars, **HYPER)
        with pytest.raises(ValueError, match="stream"):
            mok.AdamwTensors(_with(ts, grads), stream=other)
    assert _equal(_tensors(), ts)                     # nothing ran yet
    want = _tensors()
    for step in range(1, 5):
        new = _gradients(step)
        for g, n in zip(grads, new):
            g.copy_(n)
        scalars.view(torch.int32)[2] = step
        graph.replay()
        torch.cuda.synchronize()
        mok.mok_adamw_step(mok.AdamwTensors(_with(want, new)), step=step, scalars=scalars, **HYPER)
        torch.cuda.synchronize()
        assert _equal(want, ts), step
