"""Calls with stream= another stream than the current one: what they allocate has to belong to the
stream that the kernels run on (memory of the current stream's pool may still be in use there, and is
handed out again once the call has dropped it), and new outputs stay until the caller's stream is done.

Without a GPU the streams, the allocations and the library are stand-ins that write down the order."""

import contextlib

import pytest
import torch

import ternary_weight_linear_03_b200 as bl
from ternary_weight_linear_03_b200 import bitlinear as binding
from ternary_weight_linear_03_b200 import synthetic as syn

BF16, F32, I8, U8 = torch.bfloat16, torch.float32, torch.int8, torch.uint8


class FakeStream:
    device = torch.device("cpu")

    def __init__(self, handle):
        self.cuda_stream = handle


class FakeLibrary:
    """Every size is 256 bytes; every call succeeds and notes the stream it was given."""

    def __init__(self):
        self.streams = []

    def __getattr__(self, name):
        if name.endswith("_size") or name.endswith("_bytes"):
            return lambda *a: 32 if name.endswith("row_bytes") else 256

        def call(*args):
            self.streams.append(args[-1])
            return 0
        return call


@pytest.fixture
def fakes(monkeypatch):
    here, there = FakeStream(1), FakeStream(2)
    state = dict(now=here, allocated=[], kept=[], lib=FakeLibrary(), here=here, there=there)

    @contextlib.contextmanager
    def use(stream):
        before, state["now"] = state["now"], stream or state["now"]
        yield
        state["now"] = before

    def noting(fn):
        def allocate(*args, **kw):
            state["allocated"].append(state["now"])
            return fn(*args, **{k: v for k, v in kw.items() if k != "device"})
        return allocate

    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: state["now"])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    monkeypatch.setattr(torch.cuda, "device", lambda device: contextlib.nullcontext())
    monkeypatch.setattr(torch, "empty", noting(torch.empty))
    monkeypatch.setattr(torch.Tensor, "new_empty", noting(torch.Tensor.new_empty))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: state["kept"].append((t.data_ptr(), s)))
    monkeypatch.setattr(binding, "_raw_stream", lambda device: state["now"].cuda_stream)
    monkeypatch.setattr(binding, "_lib", state["lib"])
    monkeypatch.setattr(binding, "_dev", lambda t, name: t.data_ptr())
    monkeypatch.setattr(binding, "_index", lambda t, name: -1)
    return state


def _calls():
    M, N, K, E = 40, 64, 128, 2
    x, xq, scale, gamma = torch.zeros(M, K), torch.zeros(M, K, dtype=I8), torch.zeros(M), torch.zeros(1)
    packed, packedT = torch.zeros(N, K // 4, dtype=U8), torch.zeros(K, N // 4, dtype=U8)
    W, gy, acc, sums = torch.zeros(N, K), torch.zeros(M, N, dtype=BF16), torch.zeros(M, N), torch.zeros(14)
    gate, down, each = torch.zeros(E, N, K // 4, dtype=U8), torch.zeros(E, K, N // 4, dtype=U8), torch.zeros(E)
    packed3 = torch.zeros(N, 32, dtype=U8)

    def layer():
        return bl.MoeLayer(torch.zeros(E, K), gate, each, gate, each, down, each, top_k=1)

    return {
        "quantize_weights": lambda **k: bl.quantize_weights(W, **k),
        "quantize_acts": lambda **k: bl.quantize_acts(x, **k),
        "weight_abssum": lambda **k: bl.weight_abssum(W, **k),
        "quantize_weights_from_abssum": lambda **k: bl.quantize_weights_from_abssum(W, N * K, sums, **k),
        "act_absmax": lambda **k: bl.act_absmax(x, **k),
        "quantize_acts_absmax": lambda **k: bl.quantize_acts_absmax(x, scale, **k),
        "rescale": lambda **k: bl.rescale(acc, scale, gamma, **k),
        "chain_forward": lambda **k: bl.chain_forward(x, [(packed, gamma, -1)], **k),
        "pack_base3": lambda **k: bl.pack_base3(packed, **k),
        "forward_base3": lambda **k: bl.forward_base3(x, packed3, gamma, **k),
        "pack_transpose": lambda **k: bl.pack_transpose(packed, **k),
        "backward": lambda **k: bl.backward(x, gy, packedT, gamma, **k),
        "backward_quantized": lambda **k: bl.backward_quantized(xq, scale, gy, packedT, gamma, **k),
        "forward_quantized": lambda **k: bl.forward_quantized(xq, scale, packed, gamma, **k),
        "rmsnorm_quantize": lambda **k: bl.rmsnorm_quantize(x, torch.zeros(K), x, **k),
        "rmsnorm_backward": lambda **k: bl.rmsnorm_backward(x, x, torch.zeros(K), scale, **k),
        "quantize_expert_weights": lambda **k: bl.quantize_expert_weights(torch.zeros(E, N, K), **k),
        "moe_forward": lambda **k: bl.moe_forward(x, layer(), **k),
        "forward": lambda **k: bl.forward(x, packed, gamma, **k),
        "forward_noalloc": lambda **k: bl.forward_noalloc(x, packed, gamma, **k),
        "contract_i32": lambda **k: bl.contract_i32(xq, packed, **k),
    }


@pytest.mark.parametrize("name", sorted(_calls()))
def test_a_call_allocates_on_its_own_stream(name, fakes):
    here, there = fakes["here"], fakes["there"]
    out = _calls()[name](stream=there)
    out = [t for t in (out if isinstance(out, tuple) else (out,)) if t is not None]
    assert fakes["allocated"] and all(s is there for s in fakes["allocated"])
    assert fakes["lib"].streams and all(h == there.cuda_stream for h in fakes["lib"].streams)
    assert fakes["now"] is here
    for t in out:
        assert (t.data_ptr(), here) in fakes["kept"]


@pytest.mark.parametrize("name", sorted(_calls()))
def test_without_a_stream_the_current_one_is_used(name, fakes):
    _calls()[name]()
    assert all(s is fakes["here"] for s in fakes["allocated"]) and not fakes["kept"]
    assert all(h == fakes["here"].cuda_stream for h in fakes["lib"].streams)
    n = len(fakes["allocated"])
    _calls()[name](stream=fakes["here"])
    assert len(fakes["allocated"]) == 2 * n and not fakes["kept"]


def test_given_outputs_are_left_to_the_caller(fakes):
    x, y = torch.zeros(2, 128), torch.zeros(2, 64, dtype=BF16)
    bl.forward(x, torch.zeros(64, 32, dtype=U8), torch.zeros(1), y=y, stream=fakes["there"])
    assert not fakes["kept"]


def test_a_stream_of_another_device_is_refused(fakes):
    far = FakeStream(3)
    far.device = torch.device("cuda", 1)
    with pytest.raises(ValueError):
        bl.quantize_acts(torch.zeros(2, 128), stream=far)
    assert not fakes["lib"].streams


@pytest.mark.gpu
def test_results_on_a_stream_beside_the_current_one():
    """Each call runs behind a wait on a side stream; meanwhile the current stream takes memory and
    overwrites it. What the call dropped or is still to write must not be among it."""
    M, N, K, E = 40, 320, 512, 4
    x = syn.activations(M, K, 1).cuda()
    r = syn.activations(M, K, 2).cuda()
    packed, gamma = bl.quantize_weights(syn.weights(N, K, 0.02, seed=3).cuda())
    packedT, gain = bl.pack_transpose(packed), torch.ones(K, device="cuda")
    xq, scale, h, rstd = bl.rmsnorm_quantize(x, gain, r)
    gy = (torch.randn((M, N), generator=syn.gen(4)) * 0.01).bfloat16().cuda()
    W = (torch.randn((E, 3, N, K), generator=syn.gen(5)) * 0.02).cuda()
    stacks = [bl.quantize_expert_weights(W[:, i].reshape(E, *s).contiguous())
              for i, s in enumerate(((N, K), (N, K), (K, N)))]
    router = torch.randn((E, K), generator=syn.gen(6)).cuda()
    layer = bl.MoeLayer(router, *stacks[0], *stacks[1], *stacks[2], top_k=2)
    W0 = W[:, 0].contiguous()
    calls = [
        lambda **k: bl.rmsnorm_quantize(x, gain, r, **k),
        lambda **k: bl.rmsnorm_backward(x, h, gain, rstd, **k),
        lambda **k: bl.forward_quantized(xq, scale, packed, gamma, **k),
        lambda **k: bl.backward_quantized(xq, scale, gy, packedT, gamma, **k),
        lambda **k: bl.moe_forward(x, layer, **k),
        lambda **k: bl.quantize_expert_weights(W0, **k),
        lambda **k: bl.forward(x, packed, gamma, **k),
        lambda **k: bl.backward(x, gy, packedT, gamma, **k),
        lambda **k: bl.contract_i32(xq, packed, **k),
        lambda **k: bl.chain_forward(x, [(packed, gamma, -1)], **k),
        lambda **k: bl.quantize_weights(W0[0], **k),
    ]
    side, here = torch.cuda.Stream(), torch.cuda.current_stream()
    for call in calls:
        want = call()
        want = want if isinstance(want, tuple) else (want,)
        torch.cuda.synchronize()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)  # a millisecond
        got = call(stream=side)
        got = got if isinstance(got, tuple) else (got,)
        spoil = [torch.full((n,), 0xFF, dtype=U8, device="cuda")
                 for n in (512, 4096, 65536, 1 << 19, 1 << 20, 4 << 20, 16 << 20) for _ in range(3)]
        here.wait_stream(side)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        del spoil, got
    assert bl.get_device_status() == 0
