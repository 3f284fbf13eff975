"""CPU check of the stream that the runner hands to each library call (fakes of the calls): the one that its caller gives,
also where that is 0 (the legacy default stream), else the runner's own."""
import pytest

from mla_latent_kv_27_b200 import runner as R
from mla_latent_kv_27_b200 import workloads as wl

CALLS = ("mla_append_cache", "mla_absorb_query", "mla_absorb_query_early", "mla_decode_attention", "mla_output_up",
         "mla_norm_rows", "mla_quantize_rows", "mla_project_fp8", "mla_append_rows")


class Anything:
    """Stands for every attribute that the calls get."""

    def __getattr__(self, name):
        return Anything()

    def __getitem__(self, at):
        return self


class FakeLayer(R.MLALayer):
    def __init__(self, stream):
        self.stream, self.w, self.q_rank, self.n_split = stream, wl.WORKLOADS["tiny_fp32"], 48, 0

    def __getattr__(self, name):
        return Anything()


@pytest.mark.parametrize("own,given,want", [(None, None, None), (None, 0, 0), (7, None, 7), (7, 0, 0), (7, 9, 9), (0, None, 0)])
@pytest.mark.parametrize("method", ["append", "absorb", "decode", "output", "step", "layer_step"])
def test_the_given_stream_is_used(monkeypatch, method, own, given, want):
    seen = []
    for name in CALLS:
        monkeypatch.setattr(R.B, name, lambda *args: seen.append(args[-1]))
    getattr(FakeLayer(own), method)(given)
    assert seen and all(s is want or s == want and s is not None for s in seen), seen
