"""CPU-side refusals of the rotary call's rows: missing outputs, outputs whose tokens share elements."""
import pytest
import torch

from speculative_decoding_vocab_gb300 import binding as ssd

bf, i32 = torch.bfloat16, torch.int32


def call(q, q_out, **kw):
    B, S, _, d = q.shape
    ssd.ssd_tree_rope(q, None, torch.zeros(d // 2, dtype=torch.int64), d, torch.zeros(B, dtype=i32), q_out, None,
                      status=torch.zeros(1, dtype=i32), **kw)


def rows(B, S, H, d):
    return torch.zeros(B, S, H, d, dtype=bf)


def test_a_missing_output_is_named():
    with pytest.raises(ValueError, match="q_out"):
        call(rows(2, 3, 4, 64), None)
    with pytest.raises(ValueError, match="k_out"):
        ssd.ssd_tree_rope(None, rows(2, 3, 4, 64), torch.zeros(32, dtype=torch.int64), 64, torch.zeros(2, dtype=i32), None, None,
                          status=torch.zeros(1, dtype=i32))


@pytest.mark.parametrize("shape,stride", [
    ((2, 3, 4, 64), (0, 256, 64, 1)), ((2, 3, 4, 64), (768, 0, 64, 1)), ((2, 3, 4, 64), (768, 128, 64, 1)),
    ((2, 3, 4, 64), (512, 256, 64, 1)), ((2, 3, 4, 64), (256, 256, 64, 1)), ((2, 3, 4, 64), (256, 448, 64, 1)),
    ((1, 3, 4, 64), (0, 0, 64, 1)), ((3, 1, 4, 64), (0, 0, 64, 1)), ((2, 3, 1, 64), (64, 64, 64, 1)), ((2, 3, 1, 32), (70, 101, 32, 1))])
def test_outputs_that_overlap_are_refused(shape, stride):
    with pytest.raises(ValueError, match="overlap"):
        call(rows(*shape), torch.zeros(4096, dtype=bf).as_strided(shape, stride))


@pytest.mark.parametrize("shape,stride", [
    ((2, 3, 4, 64), (768, 256, 64, 1)), ((2, 3, 4, 64), (1000, 300, 64, 1)), ((2, 3, 4, 64), (256, 512, 64, 1)),
    ((1, 3, 4, 64), (0, 256, 64, 1)), ((3, 1, 4, 64), (256, 0, 64, 1)), ((1, 1, 4, 64), (0, 0, 64, 1)),
    ((2, 0, 4, 64), (0, 0, 64, 1)), ((0, 3, 4, 64), (0, 0, 64, 1)), ((2, 3, 1, 64), (64, 128, 64, 1)),
    ((3, 2, 1, 64), (64, 200, 64, 1)), ((2, 3, 1, 32), (70, 102, 32, 1))])
def test_outputs_that_do_not_overlap_are_taken(shape, stride):
    """These get as far as the device: there is none here."""
    with pytest.raises(ValueError, match="CUDA device"):
        call(rows(*shape), torch.zeros(4096, dtype=bf).as_strided(shape, stride))
    q = torch.zeros(4096, dtype=bf).as_strided(shape, (0, 0, 64, 1))  # inputs may be broadcast
    with pytest.raises(ValueError, match="CUDA device"):
        call(q, torch.zeros(4096, dtype=bf).as_strided(shape, stride))


@pytest.mark.parametrize("original", [1.0, 4.0, 6.0])
def test_frequencies_below_the_slow_border(original):
    """A context in which not even the fastest pair turns `slow` times: every pair is divided by the factor."""
    from speculative_decoding_vocab_gb300 import build
    build.build()
    turns, m = ssd.ssd_rope_frequencies(64, 10000.0, 4.0, original)
    whole, _ = ssd.ssd_rope_frequencies(64, 10000.0, 4.0)
    assert torch.equal(turns, whole) and m > 1


def test_binding_without_torchs_short_ways(monkeypatch):
    """The binding loads, and finds stream and device, where torch does not have the private calls that it prefers."""
    import importlib.util

    class Stream:
        cuda_stream = 77
    for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
        monkeypatch.delattr(torch._C, name, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev: Stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    spec = importlib.util.spec_from_file_location("speculative_decoding_vocab_gb300.binding_again", ssd.__file__)
    again = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(again)
    assert again._raw_stream(0) == 77 and again._current_device() == 3
