"""Every call works from a host thread that has made no CUDA call before, eager and under capture, and gives the bits
that the main thread's call gives."""
import dataclasses
import threading

import pytest
import torch

from mla_latent_kv_27_b200 import workloads as wl

pytestmark = pytest.mark.gpu


def in_a_thread(f):
    err = []

    def body():
        try:
            f()
        except BaseException as e:  # noqa: BLE001
            err.append(e)

    t = threading.Thread(target=body)
    t.start()
    t.join()
    if err:
        raise err[0]


@pytest.fixture(scope="module", params=["v2lite_bf16", "v3_bf16", "fp8_mtp2"])
def layer(request):
    from mla_latent_kv_27_b200.runner import MLALayer
    w = dataclasses.replace(wl.WORKLOADS[request.param], d_model=512)
    L = MLALayer(w, 768, lengths=(130, 64, 200))
    if w.cache_dtype == "fp8":
        L.fill_cache_projected()
    else:
        L.fill_cache_direct()
    L.draw_step_inputs()
    L.residual.normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    L.start = L.residual.clone()
    L.layer_step()
    L.append()
    torch.cuda.synchronize()
    return L


CALLS = {
    "append": lambda L, st: L.append(st), "absorb": lambda L, st: L.absorb(st), "decode": lambda L, st: L.decode(st),
    "output": lambda L, st: L.output(st), "layer_step": lambda L, st: L.layer_step(st),
}


def outputs(L):
    return [L.q_packed, L.o_lat, L.out, L.y, L.cache.rows]


@pytest.mark.parametrize("name", sorted(CALLS))
def test_first_call_of_a_thread(lib, layer, name):
    L = layer
    st = torch.cuda.current_stream().cuda_stream

    def once(run):
        for t in outputs(L)[:4]:
            t.zero_()
        L.residual.copy_(L.start)
        torch.cuda.synchronize()
        run(lambda: CALLS[name](L, st or torch.cuda.ExternalStream(0)))
        torch.cuda.synchronize()
        return [t.clone() for t in outputs(L)]

    want = once(lambda f: f())
    got = once(in_a_thread)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert lib.mla_check_device_error()[0] == 0


def test_first_call_of_a_thread_under_capture(lib, layer):
    L = layer
    st, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()

    def capture():
        with torch.cuda.graph(graph, stream=st):
            L.layer_step(st)

    L.residual.copy_(L.start)
    torch.cuda.synchronize()
    L.layer_step()
    torch.cuda.synchronize()
    want = L.y.clone()
    in_a_thread(capture)
    L.residual.copy_(L.start)
    L.y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(L.y, want)
