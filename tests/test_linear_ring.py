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
    return {
        "x_first": load in linear and load in tma and "cta_group::2" in _function(tma, load) and "mapa" in _function(tma, load),
        "arrive_far": arrive in linear
                      and re.search(r"fence_release_shared\(\);.*mbarrier\.arrive\.relaxed\.cluster", _function(linear, arrive), re.S) is not None
                      and "fence.release.sync_restrict::shared::cta.cluster" in tma
                      and f"{arrive}(smem_addr(&full[s]))" in linear
                      and ".release.cluster." in _function(linear, "mbar_arrive_first"),
        "wait_far": "PAIR ? ACQ_SHARED : ACQ_CTA> acq_stage" in linear and "get(acq_stage, full[s], par)" in linear
                    and "PAIR ? ACQ_CLUSTER : ACQ_CTA> acq_acc" in linear and "get(acq_acc, acc_empty[b]," in linear
                    and "mbar_wait_ring<decltype(acq)::value>" in linear
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


# a copy that never lands: every CTA that needs it gives up, and each comes to a clean end
@pytest.mark.parametrize("pair", [False, True], ids=["alone", "pair"])
def test_a_lost_copy(pair):
    rng = random.Random(8)
    how = _source()
    for _ in range(25):
        case = random_case(rng, pair)
        parts = case["tiles"] * case["blocks"] * 4
        cta = rng.randrange(2 if pair else 1)
        if rng.random() < 0.6:
            f = rng.randrange(parts // case["subs"])
            part = f % (case["blocks"] * 4 // case["subs"]) * case["subs"]
            lost = ("x", cta, f, 0)
            if part * 64 >= case["nc"]:
                continue                        # a stage without copies
        else:
            lost = ("code", cta, rng.randrange(parts // case["chunk_parts"]), 0)
        stop = Kernel(rng, lost=lost, **case, **how).run()
        assert all(stop)


# one wait that gives up early: whatever the rest does then, it ends, and nothing is written over
@pytest.mark.parametrize("pair", [False, True], ids=["alone", "pair"])
def test_a_wait_that_gives_up_early(pair):
    rng = random.Random(9)
    how = _source()
    gave_up = 0
    for _ in range(40):
        gave_up += any(Kernel(rng, **random_case(rng, pair), **how).run(early=0.002))
    assert gave_up > 20


# the kernel's abort as the model has it: a warp's lanes decide together, roles end at one barrier,
# and a CTA that gave up stays until its copies have landed
def test_the_end_is_the_source_s():
    with open(os.path.join(SRC, "linear.cu")) as f:
        text = f.read()
    body = text[text.index("k_linear_mma(const __grid_constant__"):text.index("cudaError_t codes_map")]
    assert "!abort_flag" not in body.replace("__all_sync(0xFFFFFFFFu, ok && !abort_flag)", "")
    end = body[body.index("no warp issues anything any more"):]
    assert end.index("linger()") < end.index("cluster_sync()") < end.index("tcgen05.dealloc")
