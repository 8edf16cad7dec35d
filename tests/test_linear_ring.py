"""The hand-over protocol of the linear layer's tensor-core kernel, in a model (no GPU), and
that the kernel's source is what the model takes it for."""

import os
import random
import re

import pytest

from linear_ring_model import Kernel, random_case

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_scaled_bit_bq_b200", "csrc")


def _function(text, name):
    """The text of a device function, from its name on to the closing brace at the start of a line."""
    at = text.index(name + "(")
    return text[at:text.index("\n}", at)]


def _source():
    """How linear.cu hands a pair's stages over, in the model's terms."""
    with open(os.path.join(SRC, "linear.cu")) as f:
        linear = f.read()
    with open(os.path.join(SRC, "tma.cuh")) as f:
        tma = f.read()
    load, arrive = "tma_load_2d_pair", "mbar_arrive_first_shared"
    wait = r"mbar_wait_ring<PAIR \? %s : ACQ_CTA>\(smem_addr\(&%s\)"
    return {
        "x_first": load in linear and load in tma and "cta_group::2" in _function(tma, load) and "mapa" in _function(tma, load),
        "arrive_far": arrive in linear
                      and re.search(r"fence_release_shared\(\);.*mbarrier\.arrive\.relaxed\.cluster", _function(linear, arrive), re.S) is not None
                      and "fence.release.sync_restrict::shared::cta.cluster" in tma
                      and f"{arrive}(smem_addr(&full[s]))" in linear
                      and ".release.cluster." in _function(linear, "mbar_arrive_first"),
        "wait_far": re.search(wait % ("ACQ_SHARED", r"full\[s\]"), linear) is not None
                    and re.search(wait % ("ACQ_CLUSTER", r"acc_empty\[b\]"), linear) is not None
                    and re.search(r"ACQ_SHARED\) fence_acquire_shared", _function(tma, "bool mbar_wait_ring")) is not None
                    and "fence.acquire.sync_restrict::shared::cluster.cluster" in tma
                    and ".acquire.cluster." in _function(tma, "bool mbar_try"),
    }


@pytest.mark.parametrize("pair", [False, True], ids=["alone", "pair"])
def test_hand_over(pair):
    rng = random.Random(7)
    how = _source()
    for _ in range(25):
        Kernel(rng, **random_case(rng, pair), **how).run()


# the model sees what it is there to see: each of the orderings left out shows
@pytest.mark.parametrize("left_out,shows", [("x_first", "'x', 1"), ("arrive_far", "'a', 1"), ("wait_far", "'a', 1")])
def test_the_model_sees_a_missing_ordering(left_out, shows):
    how = {"x_first": True, "arrive_far": True, "wait_far": True, left_out: False}
    if left_out == "x_first":
        how["arrive_far"] = False               # the second CTA relays its X with a CTA-scope arrival
    with pytest.raises(AssertionError, match="not ordered before the MMAs of stage 0") as e:
        Kernel(random.Random(1), pair=True, tiles=2, blocks=1, nc=256, subs=2, stages=3, chunks=2, chunk_parts=4, **how).run()
    if left_out != "x_first":
        assert shows in str(e.value)


# a ring of fewer parts than there are groups: a group comes by a slot late and its wait passes early
def test_the_model_sees_a_ring_that_is_too_short():
    with pytest.raises(AssertionError):
        for seed in range(40):
            Kernel(random.Random(seed), pair=False, tiles=4, blocks=3, nc=768, subs=1, stages=3, chunks=3, chunk_parts=2).run()
