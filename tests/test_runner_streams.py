"""A runner with a stream of its own, made and filled while another stream is current: its steps there read what was
written for them, without a synchronisation by the caller.  A sleep of some 50 ms on the current stream stands in
front of each write, so that a step that did not wait would read what was there before."""
import dataclasses

import pytest
import torch

from mla_latent_kv_27_b200 import runner as R
from mla_latent_kv_27_b200 import workloads as wl

pytestmark = pytest.mark.gpu

SLEEP = 100_000_000  # cycles


def make(name, stream):
    w = dataclasses.replace(wl.WORKLOADS[name], d_model=512)
    return R.MLALayer(w, 256, lengths=(130, 64, 200), stream=stream)


def fill(L):
    if L.w.cache_dtype == "fp8":
        L.fill_cache_projected()
    else:
        L.fill_cache_direct()


@pytest.mark.parametrize("name", ["v2lite_bf16", "fp8_mtp2"])
@pytest.mark.parametrize("as_int", [False, True])
def test_a_step_on_the_runners_own_stream(lib, monkeypatch, name, as_int):
    want = []
    L = make(name, None)
    fill(L)
    for seed in (1, 2):
        L.draw_step_inputs(seed)
        L.residual.zero_()
        L.layer_step()
        torch.cuda.synchronize()
        want += [L.y.clone(), L.cache.rows.clone()]

    stream = torch.cuda.Stream()
    plain = R.quantize_weight

    def late(w):
        torch.cuda._sleep(SLEEP)
        return plain(w)

    monkeypatch.setattr(R, "quantize_weight", late)
    L = make(name, stream.cuda_stream if as_int else stream)
    torch.cuda._sleep(SLEEP)
    fill(L)
    got = []
    for seed in (1, 2):
        torch.cuda._sleep(SLEEP)
        L.draw_step_inputs(seed)  # (behind the step before, too, which still reads the former inputs)
        with torch.cuda.stream(stream):
            L.residual.zero_()
        L.layer_step()
        with torch.cuda.stream(stream):
            got += [L.y.clone(), L.cache.rows.clone()]
    torch.cuda.synchronize()
    assert lib.mla_check_device_error()[0] == 0
    for a, b in zip(got, want):
        assert torch.equal(a, b)
