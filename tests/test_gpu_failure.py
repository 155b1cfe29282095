"""Failure detection without a GPU fault: a wait that nothing completes runs
out its bounded limit, the kernel records a device timeout in the error
word and returns, the host reads RLK_ERR_DEVICE_TIMEOUT, the word is
cleared, and the same context then runs the hot path correctly."""
import contextlib
import ctypes

import numpy as np
import pytest

import oracle
from deterministic_context_attention_gb300 import synth
from tests.gpu_helpers import lib, torch_cuda

pytestmark = pytest.mark.gpu


def test_bounded_wait_reports_timeout_and_context_survives():
    torch = torch_cuda()
    rlk = lib()
    rlk.rlk_attn_check_device_error()  # a clean error word to start from
    rlk.rlk_attn_selftest_wait_timeout()
    with pytest.raises(rlk.RlkError) as e:
        rlk.rlk_attn_check_device_error()
    assert e.value.status == 6  # RLK_ERR_DEVICE_TIMEOUT
    assert "0x7e1" in rlk.rlk_attn_last_error()
    rlk.rlk_attn_check_device_error()  # reading the word cleared it
    # the context is intact: a RoPE pass still matches the oracle bit for bit
    from deterministic_context_attention_gb300 import device as dv
    cu = synth.cu_seqlens([100, 37])
    x = synth.normal_bf16(61, synth.T_Q, (137, 8, 128))
    xd = dv.bf16_to_device(x)
    table = torch.from_numpy(rlk.rlk_attn_rope_table(1.0e6, 100)).cuda()
    rlk.rlk_attn_rope(rlk.make_params(2), xd, xd, 8, cu, None, table, 100)
    rlk.rlk_attn_check_device_error()
    pos = np.concatenate([np.arange(100), np.arange(37)]).astype(np.int32)
    np.testing.assert_array_equal(xd.float().cpu().numpy(), oracle.rope_f32(x, pos, 1.0e6))


@contextlib.contextmanager
def _invalid_capture(torch):
    """A stream whose capture a forbidden call has ended: every launch and fill on it
    comes back with an error, and nothing reaches the GPU."""
    cu = ctypes.CDLL("libcuda.so.1")
    stream = torch.cuda.Stream()
    handle, graph = ctypes.c_void_p(stream.cuda_stream), ctypes.c_void_p()
    assert cu.cuStreamBeginCapture_v2(handle, 1) == 0  # of this thread
    try:
        assert cu.cuStreamSynchronize(handle) != 0
        yield stream
    finally:
        cu.cuStreamEndCapture(handle, ctypes.byref(graph))


def _diff_calls():
    """The differential calls and the append by name, each a function of a stream, and
    what they write."""
    from tests.test_gpu_diff import Paged, Problem
    torch = torch_cuda()
    rlk = lib()
    p = Problem([150, 20], [150, 20], 8, 2, seed=51)
    dev = p.device()
    out, outb, out2, lse = p.forward(dev)
    dout = torch.from_numpy(p.dout).cuda().to(torch.bfloat16)
    ws = torch.empty(rlk.rlk_attn_workspace_size(p.params, rlk.RLK_OP_DIFF_BACKWARD, p.cq), dtype=torch.uint8, device="cuda")
    grads = [torch.empty(x.shape, device="cuda") for x in dev]
    c = Paged([700, 30], 8, 2, 16, seed=51)
    dec = c.outputs()
    dlam = torch.empty(8, device="cuda")
    lse1 = lse[..., 0].contiguous()
    plain_ws = torch.empty(rlk.rlk_attn_workspace_size(p.params, rlk.RLK_OP_BACKWARD, p.cq), dtype=torch.uint8, device="cuda")
    calls = {
        "prefill": lambda st: rlk.rlk_attn_diff_prefill(p.params, *dev, p.cq, p.ck, -1, out, outb, out2, lse, stream=st),
        "backward": lambda st: rlk.rlk_attn_diff_backward(p.params, *dev, out, out2, dout, lse, p.cq, -1, *grads, ws, stream=st),
        "empty backward": lambda st: rlk.rlk_attn_diff_backward(p.params, None, None, None, dev[3], None, None, None, None, [0, 0, 0],
                                                                -1, None, None, None, dlam, None, stream=st),
        "decode": lambda st: c.call(0, dec, stream=st),
        "append": lambda st: rlk.rlk_attn_cache_append(c.p.params, None, None, c.dev[1], None, c.dev[2], c.p.ck, None, None, 0, 128,
                                                       c.kp, c.vp, c.n_pages, 16, c.table, c.max_pages, stream=st),
        "plain backward": lambda st: rlk.rlk_attn_backward(p.params, *dev[:3], out, dout, lse1, p.cq, -1,
                                                           *grads[:3], plain_ws, stream=st),
    }
    return calls, [out, out2, lse, *grads, *dec]


def test_a_failed_launch_says_why_and_leaves_the_next_call_alone():
    torch = torch_cuda()
    rlk = lib()
    calls, outputs = _diff_calls()
    for call in calls.values():
        call(None)
    torch.cuda.synchronize()
    want = [x.clone() for x in outputs]
    for name, call in calls.items():
        with _invalid_capture(torch) as stream:
            with pytest.raises(rlk.RlkError) as e:
                call(stream)
            assert e.value.status == 7, name  # RLK_ERR_CUDA
            assert "capture" in rlk.rlk_attn_last_error(), (name, rlk.rlk_attn_last_error())
        for other, again in calls.items():
            try:
                again(None)
            except rlk.RlkError as err:
                pytest.fail(f"{other} after a failed {name}: {err}")
    rlk.rlk_attn_check_device_error()
    for x, w in zip(outputs, want):
        assert torch.equal(x, w)


@pytest.mark.parametrize("kind", [0, 1])
def test_a_refused_backward_launch_leaves_no_error_behind(kind):
    # a grid of no block, which the runtime refuses
    torch = torch_cuda()
    calls, _ = _diff_calls()
    rlk = lib()
    launch = getattr(rlk.load(), f"_ZN3rlk11launch_dbwdILi{kind}EEE9cudaErrorRKNS_9BwdParamsEiRK14CUtensorMap_stS7_S7_S7_bP11CUstream_st")
    launch.restype = ctypes.c_int
    raw = ctypes.create_string_buffer(1 << 16)  # parameters and tensor maps, all zero
    at = (ctypes.addressof(raw) + 127) // 128 * 128
    ptr = [ctypes.c_void_p(at)] + [ctypes.c_void_p(at + (1 << 15) + 128 * i) for i in range(4)]
    for overlap in (False, True):
        assert launch(ptr[0], 0, *ptr[1:], overlap, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) != 0
        calls["prefill"](None)
    rlk.rlk_attn_check_device_error()
