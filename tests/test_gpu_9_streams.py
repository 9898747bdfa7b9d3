"""Calls on a stream that is not the current one: what the binding allocates
belongs to the call's stream, so work queued on the current stream that still
uses freed memory cannot write into it; a stream of another device is refused."""
import pytest
import torch

from ultra_bit_dit_amd import lowbit as lb
from test_gpu_9_kv8 import Cache, fill, i32

pytestmark = pytest.mark.gpu


def quantize(s):
    x = torch.randn(256, 512, device="cuda").bfloat16()
    return lambda **k: lb.quantize_mxfp4(x, values=True, **k)


def product(s):
    w = lb.quantize_mxfp4(torch.randn(512, 512, device="cuda"))
    x = torch.randn(64, 512, device="cuda").bfloat16()
    return lambda **k: (lb.gemm_mxfp4(64, 512, 512, w[0], w[1], x, **k),)


def packed(s):
    codes = torch.randint(0, 256, (256, 256), device="cuda", dtype=torch.uint8)
    scales = torch.randint(100, 130, (256, 16), device="cuda", dtype=torch.uint8)
    return lambda **k: lb.pack_mxfp4(codes, scales, **k)


def attention(s):
    c = Cache([200], 16, 2, 64, seed=1)
    fill(c, [200], 2)
    table, lens = c.tables(), i32([200])
    q = torch.randn(60, 4, 64, device="cuda").bfloat16()
    return lambda **k: lb.attention_kv8(q, c.gpu, table, lens, return_lse=True, **k)


@pytest.mark.parametrize("make", [quantize, product, packed, attention])
def test_outputs_belong_to_the_calls_stream(make):
    print(f"outputs of {make.__name__} on another stream", flush=True)
    s = torch.cuda.Stream()
    call = make(s)
    want = [t.clone() for t in call()]
    call(stream=s)  # its workspace, if it needs one
    torch.cuda.synchronize()
    held = []
    for t in want:  # memory of every output's size, in use on the current stream for some time and freed
        held += [torch.empty_like(t) for _ in range(2)]
    torch.cuda._sleep(200_000_000)
    for t in held:
        t.view(torch.uint8).fill_(0x55)
    del held, t
    got = call(stream=s)
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g.view(torch.uint8), w.view(torch.uint8)), make.__name__


class OtherDevice:
    cuda_stream, device_index = 0, 1


@pytest.mark.parametrize("make", [quantize, product, packed, attention])
def test_stream_of_another_device_is_refused(make):
    print(f"{make.__name__} on a stream of another device", flush=True)
    call = make(None)
    with pytest.raises(ValueError):
        call(stream=OtherDevice())


def test_append_on_a_stream_of_another_device_is_refused():
    print("append on a stream of another device", flush=True)
    c = Cache([20], 16, 2, 64, seed=1)
    k = torch.randn(20, 2, 64, device="cuda").bfloat16()
    before = [t.clone() for t in c.gpu]
    with pytest.raises(ValueError):
        lb.kv8_append(c.gpu, c.tables(), i32([20]), k, k, stream=OtherDevice())
    torch.cuda.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(before, c.gpu))
