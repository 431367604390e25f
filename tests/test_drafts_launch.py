"""The host side of attn_tree.hip with a recorder in place of the HIP runtime, and its split rule.  No GPU
is involved."""
from test_mixers_launch import recorded


def test_tree_launches_and_splits(tmp_path):
    recorded(tmp_path, "check_tree_launch.cpp", "attn_tree.hip")
