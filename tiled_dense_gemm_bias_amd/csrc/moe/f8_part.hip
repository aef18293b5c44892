#include "gm_launch.hpp"

GBM_PART_TABLE(f8_part)
