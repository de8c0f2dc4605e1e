"""bench.py reports the GEMM's HBM traffic from a committed summary, and only
if that was measured on the current GEMM sources."""

import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import bench  # noqa: E402


def test_traffic_summary_belongs_to_the_gemm_sources():
    assert bench.read_traffic() is not None
