"""Ways of calling the operators around the experts' products: from several host threads,
under graph capture, and at the ends of their sizes."""
import ctypes
import threading

import pytest
import torch

import block_scaled_fp8_token_amd as F
from block_scaled_fp8_token_amd import _lib
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def norm_backward_into(a, d_w, stream):
    """The C entry: gradients of a norm with a branch, its weight gradients into d_w [3, N]."""
    T, N = a["h"].shape
    p = {n: t.data_ptr() for n, t in a.items()}
    return _lib.residual_rms_norm_backward(
        p["dz"], N, p["dh"], N, p["h"], N, 0, p["y"], N, p["w"], p["w"], 0, p["w"], 1.0, 1e-6, 0.0, T, N, p["dx"], N,
        p["dy"], N, d_w[0].data_ptr(), d_w[1].data_ptr(), d_w[2].data_ptr(), 0, stream)


def norm_state(seed, T, N):
    torch.manual_seed(seed)
    a = {n: torch.randn(T, N, device=DEV).to(BF) for n in ("dz", "dh", "h", "y")}
    a.update(w=torch.randn(N, device=DEV).to(BF), dx=torch.empty(T, N, dtype=BF, device=DEV),
             dy=torch.empty(T, N, dtype=BF, device=DEV))
    return a


def unused_stream():
    """A stream that no call of the library has seen (torch's own come from a pool and come again)."""
    path = next(line.split()[-1] for line in open("/proc/self/maps") if "libamdhip64" in line)
    handle = ctypes.c_void_p()
    assert ctypes.CDLL(path).hipStreamCreateWithFlags(ctypes.byref(handle), 1) == 0  # not blocking
    return torch.cuda.ExternalStream(handle.value)


def test_host_threads_on_one_stream():
    # calls whose launches share the stream's workspace: norm backward, dispatch, a split GEMM
    calls, T, N, E, M, K = 60, 300, 1024, 16, 64, 512
    states = [norm_state(s, T, N) for s in (1, 2)]
    x = torch.randn(512, K, device=DEV).to(BF)
    ids = torch.randint(0, E, (512, 4), device=DEV, dtype=torch.int32)
    qa, sfa = F.fp8_quant_group_pack(torch.randn(64, 4096, device=DEV).to(BF))
    qb, sfb = F.fp8_block_quant_128x128(torch.randn(1024, 4096, device=DEV).to(BF))
    assert F.gemm_config(F.LAYOUT_DENSE, 64, 1024, 4096)["splits"] > 1
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    grads = [torch.empty(calls, 3, N, device=DEV) for _ in states]
    slots = torch.full((calls, 512, 4), -7, dtype=torch.int32, device=DEV)
    counts = torch.empty(calls, E, dtype=torch.int32, device=DEV)
    q = torch.empty(E, M, K, dtype=torch.uint8, device=DEV)
    sf = torch.empty(E, 1, M, dtype=torch.int32, device=DEV)
    c = torch.empty(calls, 64, 1024, dtype=BF, device=DEV)
    errors = []

    def norm(i, n):
        st = norm_backward_into(states[i], grads[i][n], stream.cuda_stream)
        if st:
            errors.append(st)

    def dispatch(n):
        F.fp8_quant_group_pack_to_experts(x, ids, E, M, q=q, sf=sf, masked_m=counts[n], slot_of=slots[n], stream=stream)

    def gemm(n):
        F.fp8_block_gemm_nt(qa, sfa, qb, sfb, c=c[n], stream=stream)

    work = [lambda n: norm(0, n), lambda n: norm(1, n), dispatch, gemm]
    for fn in work:  # alone: call 0 of each, also the workspace's size
        fn(0)
    stream.synchronize()
    together = threading.Barrier(len(work))

    def many(fn):
        together.wait()
        for n in range(1, calls):
            fn(n)
    threads = [threading.Thread(target=many, args=(fn,)) for fn in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    stream.synchronize()
    assert not errors
    for got in (*grads, slots, counts, c):
        assert (got == got[:1]).all()


def test_combine_of_more_tokens_than_a_launch_takes():
    # three workgroups a token: the tokens past 2^23 workgroups are a second launch (34 GB of output)
    T, N, E, M = 1 << 22, 4104, 2, 4
    y = torch.randn(E, M, N, device=DEV).to(BF)
    pair = torch.randint(0, E * M, (T, 1), device=DEV, dtype=torch.int32)
    w = torch.randint(1, 5, (T, 1), device=DEV).float()
    out = F.moe_combine(y, pair // M, pair % M, w)
    for t in range(0, T, 1 << 18):
        rows = slice(t, t + (1 << 18))
        want = (y.view(E * M, N).float()[pair[rows, 0].long()] * w[rows]).to(BF)
        assert torch.equal(out[rows], want), "tokens from %d" % t
    del out, want
    torch.cuda.empty_cache()


def test_combine_backward_of_no_columns():
    ids = torch.zeros(3, 2, dtype=torch.int32, device=DEV)
    w = torch.ones(3, 2, device=DEV)
    y, d_out = torch.empty(2, 4, 0, dtype=BF, device=DEV), torch.empty(3, 0, dtype=BF, device=DEV)
    d_w = torch.full((3, 2), float("nan"), device=DEV)
    d_y, got = F.moe_combine_backward(d_out, y, ids, ids, w, d_weights=d_w)
    assert got is d_w and torch.equal(d_w, torch.zeros_like(d_w)) and d_y.shape == (2, 4, 0)
    _, got = F.moe_combine_backward(d_out, y, ids, ids)
    assert got is None


def test_norm_backward_of_one_row_captured_first():
    N = 1024
    a = norm_state(3, 1, N)
    want, got = torch.empty(3, N, device=DEV), torch.empty(3, N, device=DEV)
    assert norm_backward_into(a, want, torch.cuda.current_stream().cuda_stream) == 0
    rows = a["dx"].clone(), a["dy"].clone()
    torch.cuda.synchronize()
    stream, graph = unused_stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        status = norm_backward_into(a, got, stream.cuda_stream)
    assert status == 0
    for _ in range(4):
        for t in (got, a["dx"], a["dy"]):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(a["dx"], rows[0]) and torch.equal(a["dy"], rows[1])
        norm_backward_into(norm_state(4, 1, N), torch.empty(3, N, device=DEV), torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()


def binding_grads(a):
    return F.residual_rms_norm_backward(a["dz"], a["h"], a["w"], d_h=a["dh"], y=a["y"], w_post=a["w"], gate=a["w"])


def test_norm_backward_captured_on_a_stream_of_its_own():
    # the partial sums of the binding's calls come from torch's allocator, so the capture is the first call there
    a = norm_state(5, 300, 1024)
    want = [t.clone() for t in binding_grads(a)]
    torch.cuda.synchronize()
    stream, graph = unused_stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        got = binding_grads(a)
    for _ in range(4):
        for t in got:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g, w)
        binding_grads(norm_state(6, 300, 1024))
        torch.cuda.synchronize()


def test_replays_of_norm_backward_beside_calls_on_the_capture_stream():
    a, b = norm_state(7, 600, 2048), norm_state(8, 600, 2048)
    want_a, want_b = ([t.clone() for t in binding_grads(s)] for s in (a, b))
    torch.cuda.synchronize()
    stream, other, graph = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        got_a = binding_grads(a)
    for _ in range(20):
        with torch.cuda.stream(other):
            graph.replay()
        with torch.cuda.stream(stream):
            got_b = binding_grads(b)
        torch.cuda.synchronize()
        for g, w in zip((*got_a, *got_b), (*want_a, *want_b)):
            assert torch.equal(g, w)
