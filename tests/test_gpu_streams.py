"""Calls on a stream they name: what they allocate belongs to that stream.  Memory of the current
stream's pool may still be in use by work that is queued there, and may be handed to other work
there while the named stream writes it."""
import pytest
import torch

import online_softmax_forward_gb300 as pkg
from gpu_util import ensure_built

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


def pool(handle):
    """(bytes in use, bytes held) of a stream's memory."""
    segments = [s for s in torch.cuda.memory_snapshot() if s["stream"] == handle]
    return sum(s["allocated_size"] for s in segments), sum(s["total_size"] for s in segments)


def new(*s, dt=BF):
    return torch.randn(*s, device="cuda").to(dt)


def attention():
    q, k = new(1, 32, 2048, 128), new(1, 8, 300, 128)
    return lambda s: pkg.attention(q, k, k, stream=s)


def fp32_output():
    q, k = new(1, 32, 2048, 128), new(1, 8, 300, 128)
    return lambda s: pkg.attention(q, k, k, out_dtype=F, stream=s)


def blocked():
    q, k = new(8, 32, 1000, 64, dt=F), new(8, 32, 20, 64, dt=F)
    return lambda s: pkg.attention_f32_blocked(q, k, k, 32, 32, stream=s)


def splitkv():
    q, k = new(4, 32, 64, 128), new(4, 32, 2000, 128)
    return lambda s: pkg.attention_splitkv(q, k, k, n_splits=16, stream=s)  # a workspace of 68 MB


def merge():
    o, lse = new(3, 100000, 64, dt=F), new(3, 100000, dt=F)
    return lambda s: pkg.merge(o, lse, stream=s)


def merge_strided():
    o, lse = new(3, 64, 100000, dt=F).transpose(1, 2), new(3, 100000, dt=F)
    return lambda s: pkg.merge(o, lse, stream=s)


def backward():
    q, k, lse = new(1, 32, 2048, 128), new(1, 8, 300, 128), new(1, 32, 2048, dt=F)
    return lambda s: pkg.attention_bwd(q, k, k, q, lse, q, stream=s)


def rotary():
    q, rot, pos = new(1, 32, 2048, 128), pkg.Rotary(128), torch.zeros(1, 2048, dtype=torch.int32, device="cuda")
    return lambda s: pkg.rotary(q, q, rot, pos, stream=s)


@pytest.mark.parametrize("make", [attention, fp32_output, blocked, splitkv, merge, merge_strided, backward, rotary])
def test_new_tensors_belong_to_the_named_stream(make):
    ensure_built()
    call = make()
    want = call(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    del want
    torch.cuda.empty_cache()
    before = pool(torch.cuda.current_stream().cuda_stream)
    got = call(side)
    assert pool(torch.cuda.current_stream().cuda_stream) == before
    assert pool(side.cuda_stream)[0] >= sum(t.numel() * t.element_size() for t in got)
    side.synchronize()
    again = call(None)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    lib = pkg.load_test_library() if make is blocked else pkg
    assert lib.attn_check_status(None) == pkg.ATTN_OK


@pytest.mark.parametrize("make", [attention, blocked, splitkv, merge])
def test_any_object_with_a_stream_handle_names_a_stream(make):
    """These calls have taken an object that is no torch stream, for its ``cuda_stream``."""
    ensure_built()
    call, side = make(), torch.cuda.Stream()
    torch.cuda.synchronize()

    class Handle:
        cuda_stream = side.cuda_stream

    got = call(Handle())
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, call(None)))
