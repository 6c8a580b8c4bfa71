"""Calls of the transformer-block operators on a stream that is not the current one, without a
synchronisation between the two: what a call allocates is not memory that work queued on the
current stream still uses, and a result that was dropped is not reused before the work that was
queued on it."""
import pytest
import torch

pytestmark = pytest.mark.gpu
ROWS, D = 4096, 2048


def _queue_work():
    """Some milliseconds of products on the current stream."""
    a = torch.ones(4096, 4096, device="cuda") / 4096
    for _ in range(60):
        a = a @ a
    return a


def _calls(P):
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(ROWS, D, generator=g, device="cuda")
    gy = torch.randn(ROWS, D, generator=g, device="cuda")
    W = torch.randn(D, D, generator=g, device="cuda") * D ** -0.5
    v = torch.randn(D, generator=g, device="cuda")
    _, _, mean, rstd = P.pkm_layernorm_forward(x, v, v)
    return {"norm": lambda s: P.pkm_layernorm_forward(x, v, v, stream=s)[0],
            "norm with add": lambda s: P.pkm_layernorm_forward(x, v, v, add=gy, stream=s)[1],
            "norm backward": lambda s: P.pkm_layernorm_backward(gy, x, mean, rstd, v, stream=s)[0],
            "dense": lambda s: P.pkm_linear_forward(x, W, v, stream=s)[0],
            "dense pre": lambda s: P.pkm_linear_forward(x, W, v, activation="gelu", want_pre=True,
                                                        stream=s)[1]}


def test_results_take_no_memory_that_queued_work_uses():
    import product_key_memory_b200 as P
    for name, call in _calls(P).items():
        want = call(None)
        side = torch.cuda.Stream()
        call(side)                                     # the stream's pool has been used before
        torch.cuda.synchronize()
        t = torch.full((ROWS, D), 3.0, device="cuda")  # as large as the result
        _queue_work()
        copy = t.clone()                               # queued behind it
        del t
        got = call(side)
        torch.cuda.synchronize()
        assert bool((copy == 3.0).all()), name
        assert torch.equal(got, want), name


def test_a_dropped_result_is_not_reused_before_its_readers():
    import product_key_memory_b200 as P
    for name, call in _calls(P).items():
        want = call(None)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        got = call(side)
        torch.cuda.current_stream().wait_stream(side)
        _queue_work()
        copy = got.clone()                             # on the current stream
        del got
        with torch.cuda.stream(side):
            other = torch.full((ROWS, D), 5.0, device="cuda")
        torch.cuda.synchronize()
        assert torch.equal(copy, want), name
        assert bool((other == 5.0).all()), name


def test_the_current_stream_and_device_are_as_they_were():
    import product_key_memory_b200 as P
    before = torch.cuda.current_stream()
    call = _calls(P)["dense"]
    call(torch.cuda.Stream())
    assert torch.cuda.current_stream() == before and torch.cuda.current_device() == 0
    x = torch.ones(4, 8, device="cuda")
    with pytest.raises(P.PKMError):                    # refused inside the call: unaligned
        flat = torch.ones(33, device="cuda")
        P.pkm_layernorm_forward(flat[1:].view(4, 8), x[0], None, stream=torch.cuda.Stream())
    assert torch.cuda.current_stream() == before
