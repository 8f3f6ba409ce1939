"""The kernels that are launched while the kernel in front of them ends (the
rotating append, the FP8 append and the FP8 decode): whatever that kernel still
writes is read after it."""

import ctypes
import re

import pytest
import torch

import paged_kv_cache_386_b200 as pkv
from paged_kv_cache_386_b200 import build as pkv_build


def test_inputs_are_not_read_through_the_read_only_path():
    """ld.global.nc (__ldg, restrict-qualified kernel arguments) is undefined for memory written after a kernel's start."""
    for name in ("pkv_append_f8.cuh", "pkv_decode_f8.cuh"):
        code = re.sub(r"//[^\n]*", "", (pkv_build.CSRC / name).read_text())
        assert not re.findall(r"__ldg|__restrict__|\.nc\b", code), name
        for kernel in re.findall(r"__global__[^{]*?(pkv_\w+_kernel)\(", code):
            if kernel != "pkv_copy_blocks_f8_kernel":  # launched in the ordinary way
                assert "wait_for_kernel_before();" in code.split(kernel + "(", 1)[1].split("__global__")[0], kernel


def rows(shape, g, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g).to(dtype).cuda()


class Inputs:
    """A step of three sequences (head_dim 128, 4 query heads to a kv head), every input a tensor of its own."""

    def __init__(self):
        g = torch.Generator().manual_seed(71)
        self.t = dict(q=rows((3, 8, 128), g), k=rows((3, 2, 128), g), v=rows((3, 2, 128), g),
                      pos=torch.tensor([37, 16, 900]).cuda(), slots=torch.tensor([3 * 16 + 5, 7 * 16, 60 * 16 + 4]).cuda(),
                      table=pkv.rotary_table(1024, 128), lens=torch.tensor([38, 17, 901], dtype=torch.int32).cuda(),
                      tables=torch.stack([torch.randperm(70, generator=g)[:57] for _ in range(3)]).int().cuda(),
                      kc=rows((70, 2, 16, 128), g), vc=rows((70, 2, 16, 128), g),
                      codes=torch.randint(0, 0x70, (70, 2, 2, 16, 128), generator=g, dtype=torch.uint8).cuda(),
                      scales=(2.0 ** torch.randint(-9, -4, (70, 2, 2), generator=g)).cuda())
        # In range, and nothing like what comes.
        self.before = dict(pos=1, slots=-1, lens=0, tables=69, table=0.5, scales=1.0)

    def copies(self):
        return {n: t.clone() for n, t in self.t.items()}


def append_rope(t):
    return [pkv.paged_kv_append_rope(t["k"], t["v"], t["pos"], t["table"], t["slots"], t["kc"], t["vc"], q=t["q"]),
            t["kc"], t["vc"]]


def append_fp8(t):
    pkv.paged_kv_append_fp8(t["k"], t["v"], t["slots"], t["codes"].view(torch.float8_e4m3fn), t["scales"])
    return [t["codes"], t["scales"]]


def append_rope_fp8(t):
    return [pkv.paged_kv_append_rope_fp8(t["k"], t["v"], t["pos"], t["table"], t["slots"],
                                         t["codes"].view(torch.float8_e4m3fn), t["scales"], q=t["q"]),
            t["codes"], t["scales"]]


def decode(t):
    return [pkv.paged_attention_decode_fp8(t["q"], t["codes"].view(torch.float8_e4m3fn), t["scales"], t["tables"],
                                           t["lens"], 0.1)]


READS = [(append_rope, ("q", "k", "v", "pos", "slots", "table", "kc", "vc")), (append_fp8, ("k", "v", "slots", "codes", "scales")),
         (append_rope_fp8, ("q", "k", "v", "pos", "slots", "table", "codes", "scales")),
         (decode, ("q", "codes", "scales", "tables", "lens"))]


@pytest.mark.gpu
@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("call,late", [(c, n) for c, names in READS for n in names])
def test_an_input_that_the_kernel_in_front_writes_last(call, late, captured):
    """The kernel in front sums up a gigabyte whose result is the input."""
    inputs = Inputs()
    want = [x.clone() for x in call(inputs.copies())]
    t = inputs.copies()
    value = t[late].clone()
    terms = torch.zeros((value.numel(), (1 << 30) // (value.numel() * value.element_size())), dtype=value.dtype, device="cuda")
    terms[:, 0] = value.flatten()

    def both():
        torch.sum(terms, 1, dtype=value.dtype, out=t[late].view(-1))
        return call(t)

    if captured:
        both()  # what the first use of an entry point or of the sum sets up
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = both()
    for _ in range(3):
        for n, x in inputs.t.items():
            t[n].copy_(x)
        t[late].fill_(inputs.before.get(late, 0))
        torch.cuda.synchronize()
        if captured:
            graph.replay()
        else:
            got = both()
        torch.cuda.synchronize()
        for x, y in zip(got, want, strict=True):
            assert torch.equal(x, y)
    assert pkv.pkv_get_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("call,late", [(append_rope, "slots"), (append_fp8, "v"), (append_rope_fp8, "pos"), (decode, "lens"),
                                       (decode, "codes")])
def test_an_input_from_another_stream(call, late, captured):
    """The input is summed up on another stream; a short kernel and the wait for that stream stand in front of the call."""
    inputs = Inputs()
    want = [x.clone() for x in call(inputs.copies())]
    t = inputs.copies()
    value = t[late].clone()
    terms = torch.zeros((value.numel(), (1 << 30) // (value.numel() * value.element_size())), dtype=value.dtype, device="cuda")
    terms[:, 0] = value.flatten()
    side, short = torch.cuda.Stream(), torch.zeros(8, device="cuda")

    def both():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            torch.sum(terms, 1, dtype=value.dtype, out=t[late].view(-1))
        short.add_(1)
        main.wait_stream(side)
        return call(t)

    both()
    torch.cuda.synchronize()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = both()
    for _ in range(3):
        for n, x in inputs.t.items():
            t[n].copy_(x)
        t[late].fill_(inputs.before.get(late, 0))
        torch.cuda.synchronize()
        if captured:
            graph.replay()
        else:
            got = both()
        torch.cuda.synchronize()
        for x, y in zip(got, want, strict=True):
            assert torch.equal(x, y)
    assert pkv.pkv_get_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("call", ["append_rope", "append_fp8", "append_rope_fp8", "decode", "decode_workspace", "decode_16"])
def test_a_launch_that_fails_is_that_calls_error_alone(call):
    """A call on a stream whose capture was given up fails; the next call, elsewhere, does not."""
    rt = ctypes.CDLL("libcudart.so.12")
    t = Inputs().copies()
    fp8, q_out = t["codes"].view(torch.float8_e4m3fn), torch.empty_like(t["q"])
    ws = None
    if call == "decode_workspace":
        ws = pkv.new_workspace(pkv.paged_attention_fp8_workspace_size(3, 1, 8, 2, 128))
    elif call == "decode_16":
        ws = pkv.new_workspace(pkv.paged_attention_workspace_size(3, 8, 2, 128, torch.bfloat16))
    calls = {
        "append_rope": lambda s: pkv.paged_kv_append_rope(t["k"], t["v"], t["pos"], t["table"], t["slots"], t["kc"], t["vc"],
                                                          q=t["q"], q_out=q_out, stream=s),
        "append_fp8": lambda s: pkv.paged_kv_append_fp8(t["k"], t["v"], t["slots"], fp8, t["scales"], stream=s),
        "append_rope_fp8": lambda s: pkv.paged_kv_append_rope_fp8(t["k"], t["v"], t["pos"], t["table"], t["slots"], fp8,
                                                                  t["scales"], q=t["q"], q_out=q_out, stream=s),
        "decode": lambda s: pkv.paged_attention_decode_fp8(t["q"], fp8, t["scales"], t["tables"], t["lens"], 0.1, out=q_out,
                                                           workspace=ws, stream=s),
        "decode_16": lambda s: pkv.paged_attention_decode(t["q"], t["kc"], t["vc"], t["tables"], t["lens"], 0.1, out=q_out,
                                                          workspace=ws, stream=s)}
    calls["decode_workspace"] = calls["decode"]
    calls[call](None)
    src, dst = (torch.tensor([i], dtype=torch.int32).cuda() for i in (1, 2))
    torch.cuda.synchronize()
    stream, graph = ctypes.c_void_p(), ctypes.c_void_p()
    assert rt.cudaStreamCreateWithFlags(ctypes.byref(stream), 1) == 0
    try:
        assert rt.cudaStreamBeginCapture(stream, 2) == 0  # relaxed: nothing else is held back
        assert rt.cudaStreamSynchronize(stream) != 0      # not allowed in a capture, which ends it
        with pytest.raises(pkv.PagedKVError) as e:
            calls[call](stream.value)
        assert e.value.status == 4
    finally:
        rt.cudaStreamEndCapture(stream, ctypes.byref(graph))
        rt.cudaStreamDestroy(stream)
        rt.cudaGetLastError()
    pkv.paged_kv_copy_blocks_fp8(fp8, t["scales"], src, dst)
    pkv.paged_kv_append(t["k"], t["v"], t["slots"], t["kc"], t["vc"])
    calls[call](None)
    torch.cuda.synchronize()
    assert pkv.pkv_get_device_error() == 0
