"""The committed rocprofv3 summary of the model-side operators was taken from the
current kernel sources: the sha256 recorded beside it equals theirs now."""
import json
import os

from ring_allreduce_reduction_02_amd import profsum

PROFILES = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "profiles")


def test_profile_matches_the_sources():
    r = json.load(open(os.path.join(PROFILES, "model_operators_sources.json")))
    assert os.path.exists(os.path.join(PROFILES, r["summary"]))
    assert {"cc_sort.hip", "cc_embed.hip", "cc_route.hip", "cc_ffn.hip", "cc_ffn_rule.h"} <= set(r["kernel_sources"])
    assert r["kernel_source_sha256_16"] == profsum.sources_hash(r["kernel_sources"]), \
        "the kernels' sources changed since they were profiled"
