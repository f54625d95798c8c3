"""The configuration object holds its fields and nothing else, before and after calls."""
import copy
import ctypes

import routed_expert_ffn_renorm_b200 as moe


def test_calls_leave_the_configuration_as_it_was():
    cfg = moe.MoEConfig(hidden=256, n_routed_experts=8, moe_intermediate_size=128, num_experts_per_tok=2, topp=0.5)
    fields = dict(vars(cfg))
    size = moe.workspace_bytes(cfg, 16)
    assert vars(cfg) == fields
    again = moe.MoEConfig(**vars(cfg))  # as a config file is written and read back
    assert again == cfg and moe.workspace_bytes(again, 16) == size
    wider = copy.copy(cfg)
    wider._c().hidden = 512  # a call's argument block is its own
    assert bytes(cfg._c()) == bytes(again._c()) and ctypes.sizeof(cfg._c()) == 32
