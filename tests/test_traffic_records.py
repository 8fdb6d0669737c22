"""The committed records of the decode kernels' memory traffic belong to the sources that are built: the benchmark reports
a record only while none of the files that its kernel is compiled from has changed."""
import pytest

import bench


@pytest.mark.parametrize("layout,coder", [("lanes", "huffman"), ("lanes", "rans"), ("chunks", "huffman")])
def test_record_holds(layout, coder):
    assert bench.recorded_traffic("block_8b", layout, coder) is not None
