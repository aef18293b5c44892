#include "gx_launch.hpp"

GBX_GRAD_TABLE(wgrad_tn, EPI_GRAD)
GBX_GRAD_TABLE(part_tn, EPI_PART)
