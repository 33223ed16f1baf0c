"""What the kernel sources must not hold."""
import os
import re

import ppo_policy_loss_gb300._build as build


def test_no_tile_load_into_other_ctas_of_a_cluster():
    """The library may be used on several GPUs, so no tile load, on or off,
    writes the shared memory of a cluster's other CTAs, and no commit arrives there."""
    for name in os.listdir(build.CSRC):
        with open(os.path.join(build.CSRC, name), encoding="utf-8") as f:
            assert not re.search(r"multicast::cluster|RLG_CLUSTER", f.read()), name
