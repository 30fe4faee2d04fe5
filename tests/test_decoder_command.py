"""The decoder's command and configuration, on the CPU."""
from __future__ import annotations

import sys

import pytest
import torch

from stream_gated_residual_gb300 import decoder
from stream_gated_residual_gb300.decoder import Config


class Started(Exception):
    pass


@pytest.fixture()
def started(monkeypatch):
    """The configuration that the command would run: the model's constructor raises it."""
    def stop(cfg, **kw):
        raise Started(cfg)
    monkeypatch.setattr(decoder, "Decoder", stop)


def test_a_program_with_flags_of_its_own_can_call_it(started, monkeypatch):
    """Without arguments it runs the plain model, whatever the program's own command line says."""
    monkeypatch.setattr(sys, "argv", ["train.py", "--steps", "10"])
    with pytest.raises(Started) as e:
        decoder.main()
    assert e.value.args[0] == Config()


def test_flags(started):
    with pytest.raises(Started) as e:
        decoder.main(["--d-ff", "256", "--fp8"])
    assert e.value.args[0] == Config(d_ff=256, fp8=True)
    with pytest.raises(SystemExit):
        decoder.main(["--steps", "10"])


@pytest.mark.parametrize("bad", [
    dict(fp8=True), dict(fp8=True, d_ff=256, dtype=torch.float32), dict(fp8=True, d_ff=264), dict(fp8=True, d_ff=256, d_model=72),
    dict(d_ff=-8), dict(d_ff=100), dict(d_ff=256, activation="relu")])
def test_a_configuration_that_cannot_run_is_refused(bad):
    """Where it is made, not at the first prompt."""
    with pytest.raises(ValueError):
        Config(**bad)


@pytest.mark.parametrize("good", [
    dict(), dict(dtype=torch.float32), dict(d_ff=136, activation="gelu"), dict(d_ff=8, dtype=torch.float32),
    dict(d_ff=272, fp8=True)])
def test_configurations_that_run(good):
    Config(**good)


def test_fp8_without_feed_forward_sublayers_is_refused_by_the_command(started):
    with pytest.raises(SystemExit):
        decoder.main(["--fp8"])
